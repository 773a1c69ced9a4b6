"""rms_norm, rms_norm_backward and quantize_rows on the GPU against float64.

Tolerances, with u = 2^-24.  A sum of squares adds at most 32 terms a thread, 5 times across a warp and 16 times
across warps, so it is off by 54 u of itself (all terms are positive); the mean and eps add 2 u, the root halves
that, root and division add 2 u: 1 / rms is off by 30 u, y by 32 u of itself, plus the output's rounding.  The
scale is off by 33 u (a division); a code's argument, at most 127, by 70 u of itself, so a code is within
0.5 + 127 * 70 u of the exact quotient.  The backward pass's row sum is off by 55 u times the sum of absolute
terms; dw adds N / parts + parts / 32 + 10 times."""
import numpy as np
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


def rows(seed, N, H, dt, pad=0, first=0, size=1.0):
    """Random rows inside a buffer of NaN: `pad` elements behind each, `first` before the first one."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    buf = torch.full((first + N * (H + pad),), float("nan"), dtype=dt, device=DEV)
    x = buf[first:].as_strided((N, H), (H + pad, 1))
    x.copy_(torch.randn(N, H, generator=g, device=DEV) * size)
    return x


def step(dt):
    return torch.finfo(dt).eps / 2, torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def near(got, want, tol, dt=torch.float32):
    rel, least = step(dt)
    err = (got.double() - want).abs()
    bound = tol + rel * (want.abs() + tol) + least
    assert torch.isfinite(got).all() and (err <= bound).all(), (err / bound).max().item()


def check_codes(q, scale, y):
    want, s = head.quantize(y)
    near(scale, s, 33 * U * s)
    assert ((q.double() - want).abs() <= 0.5 + 127 * 70 * U).all()
    assert q.abs().amax() <= 127


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("N,H", [(1, 1), (1, 8), (2, 33), (3, 64), (5, 257), (7, 1024), (2, 2048), (3, 2051), (9, 4096),
                                 (2, 5120), (3, 8192), (2, 8193), (2, 16384), (2, 16383), (300, 40)])
def test_norm_sizes(tsa, dt, N, H):
    x, w = rows(N + H, N, H, dt), rows(1, 1, H, dt)[0]
    r = rows(N, N, H, dt, size=3.0)
    s = head.add_residual(x, r)
    y, rstd = head.rms_norm(s, w, 1e-6)
    a = tsa.rms_norm(x, w, residual=r)
    assert torch.equal(a.residual, s) and a.scale is None
    near(a.rstd, rstd, 30 * U * rstd)
    near(a.out, y, 32 * U * y.abs(), dt)
    b = tsa.rms_norm(x, w, residual=r, quantize=True)
    assert torch.equal(b.residual, s) and torch.equal(b.rstd, a.rstd)
    check_codes(b.out, b.scale, y)
    y, _ = head.rms_norm(x, w, 1e-6)
    c = tsa.rms_norm(x, w)
    assert c.residual is None
    near(c.out, y, 32 * U * y.abs(), dt)
    check_codes(*tsa.quantize_rows(x), x)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("pad,first", [(0, 0), (8, 0), (16, 8), (1, 0), (3, 1), (0, 1)])
def test_norm_strides_and_weights(tsa, dt, pad, first):
    N, H = 6, 1040
    x, r, w = rows(1, N, H, dt, pad, first), rows(2, N, H, dt, pad + 8, first), rows(3, 1, H, torch.float32)[0]
    out, res = rows(4, N, H, dt, pad + 3, first + 1), rows(5, N, H, dt, pad, first)
    s = head.add_residual(x, r)
    y, _ = head.rms_norm(s, w, 1e-5)
    a = tsa.rms_norm(x, w, residual=r, eps=1e-5, out=out, residual_out=res)
    assert a.out is out and a.residual is res and torch.equal(res, s)
    near(out, y, 32 * U * y.abs(), dt)
    behind = out.as_strided((N - 1, pad + 3), (H + pad + 3, 1), out.storage_offset() + H)
    assert torch.isnan(behind).all()
    q = torch.full((N, H + 5), 99, dtype=torch.int8, device=DEV)
    b = tsa.rms_norm(x, w, residual=r, eps=1e-5, quantize=True, out=q[:, 1:H + 1], residual_out=r)  # over the residual
    assert torch.equal(r, s) and (q[:, 0] == 99).all() and (q[:, H + 1:] == 99).all()
    check_codes(b.out, b.scale, y)
    y, _ = head.rms_norm(x, w, 1e-5)
    kept = x.clone()
    tsa.rms_norm(x, w, eps=1e-5, out=x)  # over the rows
    near(x, y, 32 * U * y.abs(), dt)
    codes, scale = tsa.quantize_rows(kept, out=q[:, :H])
    check_codes(codes, scale, kept)
    assert (q[:, H + 1:] == 99).all()


def test_norm_special_rows(tsa):
    x = rows(1, 6, 96, torch.float32)
    x[0], x[1] = 0.0, 0.0
    x[1, 5] = 1e-30
    x[2] *= 1e15
    x[3, 7], x[4, 9] = float("inf"), float("nan")
    w = torch.ones(96, device=DEV)
    a = tsa.rms_norm(x, w, quantize=True)
    y, _ = head.rms_norm(x, w, 1e-6)
    good = [0, 1, 2, 5]
    check_codes(a.out[good], a.scale[good], y[good])
    assert a.scale[0] == 0 and (a.out[0] == 0).all()
    assert torch.isnan(a.scale[3:5]).all() and (a.out[3:5] == 0).all()
    q, scale = tsa.quantize_rows(x)
    check_codes(q[good], scale[good], x[good])
    assert torch.isnan(scale[3:5]).all() and q[1, 5] == 127
    tiny = torch.full((2, 40), 2.0 ** -140, device=DEV)
    tiny[:, ::2] *= -0.5
    q, scale = tsa.quantize_rows(tiny)
    assert (q[:, 1::2] == 127).all() and (q[:, ::2] == -64).all()  # -63.5, ties to even
    assert torch.isnan(tsa.rms_norm(x, w).out[4]).any()
    assert torch.isnan(tsa.rms_norm(x[:1], w, eps=0.0).out).all()


def check_back(tsa, g, x, w, gr, dx=None, parts=300):
    N, H = x.shape
    rstd = head.rms_norm(x, w, 1e-6)[1].float()
    want, dw, h, f = head.rms_norm_backward(g, x, w, rstd, gr)
    got = tsa.rms_norm_backward(g, x, w, rstd, grad_residual=gr, grad_x=dx)
    r = rstd.double()[:, None]
    mean = (f * h).abs().mean(-1, keepdim=True)
    tol = r * U * (2 * f.abs() + h.abs() * 60 * mean) + 3 * U * (want.abs() + r * f.abs() + r * h.abs() * mean)
    near(got[0], want, tol, x.dtype)
    adds = N / min(N, parts) + parts / 32 + 12
    near(got[1], dw, (adds + 2) * U * (g.double() * h).abs().sum(0), w.dtype)
    return got


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("N,H", [(1, 1), (1, 16), (3, 33), (5, 256), (130, 64), (7, 1024), (9, 2051), (700, 2048),
                                 (3, 5120), (2, 8193), (4, 16384), (1000, 24)])
def test_norm_backward(tsa, dt, N, H):
    g, x, w = rows(1, N, H, dt, size=0.1), rows(2, N, H, dt), rows(3, 1, H, dt)[0]
    check_back(tsa, g, x, w, None)
    gr = rows(4, N, H, dt)
    a = check_back(tsa, g, x, w, gr)
    rstd = head.rms_norm(x, w, 1e-6)[1].float()
    b = tsa.rms_norm_backward(g, x, w, rstd, grad_residual=gr)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("pad,first", [(8, 8), (1, 0), (3, 5)])
def test_norm_backward_strides_and_in_place(tsa, dt, pad, first):
    N, H = 21, 520
    g, x, w = rows(1, N, H, dt, pad, first), rows(2, N, H, dt, pad + 8), rows(3, 1, H, torch.float32)[0]
    gr = rows(4, N, H, dt, pad)
    rstd = head.rms_norm(x, w, 1e-6)[1].float()
    want = tsa.rms_norm_backward(g, x, w, rstd, grad_residual=gr)
    assert want[1].dtype == torch.float32
    check_back(tsa, g, x, w, gr, dx=rows(6, N, H, dt, pad + 1))
    dw = torch.empty(H, device=DEV)
    over = gr.as_strided(gr.shape, gr.stride())
    got = tsa.rms_norm_backward(g, x, w, rstd, grad_residual=gr, grad_x=over, grad_weight=dw)
    assert torch.equal(got[0], want[0]) and got[1] is dw and torch.equal(dw, want[1])


def test_norm_of_many_rows(tsa):
    x, r = rows(1, 20000, 256, torch.bfloat16), rows(2, 20000, 256, torch.bfloat16)
    w = rows(3, 1, 256, torch.bfloat16)[0]
    y, _ = head.rms_norm(head.add_residual(x, r), w, 1e-6)
    near(tsa.rms_norm(x, w, residual=r).out, y, 32 * U * y.abs(), torch.bfloat16)
    check_back(tsa, r, x, w, None)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("H", [2056, 5120, 6152, 8192, 16384])
def test_many_long_rows(tsa, dt, H):
    """Rows that go through shared memory, with strides, over their inputs, and with a wider weight."""
    N = 700
    x, r, w = rows(1, N, H, dt, 8), rows(2, N, H, dt, 24, 8), rows(3, 1, H, torch.float32)[0]
    s = head.add_residual(x, r)
    y, rstd = head.rms_norm(s, w, 1e-6)
    kept = r.clone()
    a = tsa.rms_norm(x, w, residual=r, residual_out=r)
    assert torch.equal(r, s)
    near(a.rstd, rstd, 30 * U * rstd)
    near(a.out, y, 32 * U * y.abs(), dt)
    b = tsa.rms_norm(x, w, residual=kept, quantize=True)
    assert torch.equal(b.residual, s) and torch.equal(b.rstd, a.rstd)
    check_codes(b.out, b.scale, y)
    y, _ = head.rms_norm(x, w, 1e-6)
    near(tsa.rms_norm(x, w).out, y, 32 * U * y.abs(), dt)
    check_back(tsa, kept, x, w, None)
    check_back(tsa, kept, x, w, r)
    a = tsa.rms_norm_backward(kept, x, w, b.rstd, grad_residual=r)
    c = tsa.rms_norm_backward(kept, x, w, b.rstd, grad_residual=r, grad_x=kept)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1]) and tsa.device_status() == 0


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("N", [608, 2500])
@pytest.mark.parametrize("H,pad,first", [(512, 1, 1), (513, 0, 0), (1001, 0, 3), (1001, 4, 1), (2064, 1, 5), (2064, 8, 1), (4881, 0, 0),
                                         (6145, 7, 7), (8193, 0, 2), (12345, 0, 0), (16377, 0, 1), (16383, 0, 1)])
def test_many_rows_that_start_anywhere(tsa, dt, N, H, pad, first):
    """Rows whose starts lie at every place of 16 bytes, alike in each tensor: what is next to a row (NaN here) neither
    counts nor is written."""
    x, r, g = (rows(i, N, H, dt, pad, first) for i in (1, 2, 3))
    out, res, dx = (rows(i, N, H, dt, pad, first) for i in (4, 5, 6))
    w = rows(7, 1, H, dt)[0]
    codes = torch.full((first + N * (H + pad),), 99, dtype=torch.int8, device=DEV)
    q = codes[first:].as_strided((N, H), (H + pad, 1))
    s = head.add_residual(x, r)
    y, rstd = head.rms_norm(s, w, 1e-6)
    a = tsa.rms_norm(x, w, residual=r, out=out, residual_out=res)
    assert torch.equal(res, s)
    near(a.rstd, rstd, 30 * U * rstd)
    near(out, y, 32 * U * y.abs(), dt)
    b = tsa.rms_norm(x, w, residual=r, quantize=True, out=q, residual_out=res)
    assert torch.equal(res, s) and torch.equal(b.rstd, a.rstd)
    check_codes(q, b.scale, y)
    # up to eight parts of dw an SM, two rows each: N / parts + parts / 32 + 10 adds
    parts = 152 * min(8, N // 304)
    check_back(tsa, g, x, w, None, dx=dx, parts=parts)
    check_back(tsa, g, x, w, r, dx=dx, parts=parts)
    for t, beside in ((out, torch.isnan), (res, torch.isnan), (dx, torch.isnan), (q, lambda v: v == 99)):
        buf = t.as_strided((t.storage_offset() + N * (H + pad),), (1,), 0)
        assert beside(buf[:first]).all() and beside(buf[first:].view(N, H + pad)[:, H:]).all()
    kept = tsa.rms_norm_backward(g, x, w, a.rstd, grad_residual=r, grad_x=dx)
    over = tsa.rms_norm_backward(g, x, w, a.rstd, grad_residual=r, grad_x=g)
    assert torch.equal(over[0], kept[0]) and torch.equal(over[1], kept[1])
    y, _ = head.rms_norm(x, w, 1e-6)
    tsa.rms_norm(x, w, out=x)
    near(x, y, 32 * U * y.abs(), dt)
    assert tsa.device_status() == 0


def test_norm_of_more_elements_than_32_bits_count(tsa):
    N, H = 132_000, 16384
    x = torch.empty(N, H, dtype=torch.bfloat16, device=DEV)
    x[-64:] = rows(1, 64, H, torch.bfloat16)
    x[:-64] = x[-64:].repeat(N // 64, 1)[:N - 64]
    w = rows(2, 1, H, torch.bfloat16)[0]
    assert x.numel() > 2 ** 31
    a = tsa.rms_norm(x, w)
    y, _ = head.rms_norm(x[-64:], w, 1e-6)
    near(a.out[-64:], y, 32 * U * y.abs(), torch.bfloat16)
    dx, _ = tsa.rms_norm_backward(x, x, w, a.rstd, grad_x=a.out)
    want, few = tsa.rms_norm_backward(x[-64:], x[-64:], w, a.rstd[-64:])
    assert torch.equal(dx[-64:], want)


def test_norm_of_no_rows(tsa):
    x, w = torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV)
    assert tsa.rms_norm(x, w, quantize=True).out.shape == (0, 64)
    dx, dw = tsa.rms_norm_backward(x, x, w, torch.empty(0, device=DEV), grad_weight=torch.ones(64, device=DEV))
    assert dx.shape == (0, 64) and (dw == 0).all()
    assert tsa.quantize_rows(x)[0].shape == (0, 64)


def test_norm_versions_streams_and_graphs(tsa):
    x, r, w = rows(1, 33, 512, torch.bfloat16), rows(2, 33, 512, torch.bfloat16), rows(3, 1, 512, torch.bfloat16)[0]
    out, before = torch.empty_like(x), x._version
    want = tsa.rms_norm(x, w, residual=r, quantize=True)
    tsa.rms_norm(x, w, out=out)
    assert out._version == 1 and x._version == before
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = tsa.rms_norm(x, w, residual=r, quantize=True)
        back = tsa.rms_norm_backward(x, r, w, a.rstd)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want.out) and torch.equal(a.scale, want.scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = tsa.rms_norm(x, w, residual=r, quantize=True)
        gb = tsa.rms_norm_backward(x, r, w, a.rstd)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.out, want.out) and torch.equal(gb[0], back[0]) and torch.equal(gb[1], back[1])
    x.mul_(2.0)
    graph.replay()
    want = tsa.rms_norm(x, w, residual=r, quantize=True)
    assert torch.equal(b.out, want.out) and torch.equal(b.residual, want.residual)


def test_norm_refusals(tsa):
    x, w = torch.ones(4, 64, device=DEV), torch.ones(64, device=DEV)
    for call in (lambda: tsa.rms_norm(x.t(), w), lambda: tsa.rms_norm(x, w[:32]), lambda: tsa.rms_norm(x, w.half()),
                 lambda: tsa.rms_norm(x, w, residual=x.half()), lambda: tsa.rms_norm(x, w, residual_out=x),
                 lambda: tsa.rms_norm(x, w, out=x.half()), lambda: tsa.rms_norm(x, w, quantize=True, out=x),
                 lambda: tsa.rms_norm(x.long(), w), lambda: tsa.quantize_rows(x[0]),
                 lambda: tsa.rms_norm_backward(x, x, w, w), lambda: tsa.rms_norm_backward(x[:2], x, w, x[:, 0]),
                 lambda: tsa.rms_norm_backward(x, x, w, torch.ones(4, device=DEV), grad_weight=w.half())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: tsa.rms_norm(x, w, eps=-1.0), lambda: tsa.rms_norm(x[:1].expand(4, 64), w),
                 lambda: tsa.rms_norm(x, w, residual=x.clone(), out=x, residual_out=x)):
        with pytest.raises(tsa.TSAError):
            call()
