"""Host-side argument validation of the calls around the vocabulary head (no GPU work): the documented status
comes back before anything is launched, and empty calls launch nothing."""
import ctypes

import pytest
import torch

from tests.test_abi import FAKE, S

P = ctypes.c_void_p
OTHER, ODD1, ODD2, ODD4, ODD8 = P(0x20000), P(0x30001), P(0x30002), P(0x30004), P(0x30008)


@pytest.fixture(scope="module")
def lib():
    from top_sampling_apply_gb300 import _build

    _build.build()
    import top_sampling_apply_gb300 as tsa

    return tsa.load_library()


def norm(lib, x=FAKE, dt=2, N=2, H=64, xs=64, w=FAKE, wdt=2, r=None, rs=64, eps=1e-6, q=0, out=OTHER, os=64,
         scale=None, res=None, ress=64, rstd=None):
    return lib.tsa_rms_norm(x, dt, N, H, xs, w, wdt, r, rs, eps, q, out, os, scale, res, ress, rstd, None)


def test_rms_norm_validation(lib):
    for kw in ({"dt": 3}, {"wdt": 1}, {"dt": 0, "wdt": 2}):
        assert norm(lib, **kw) == S["TSA_ERR_DTYPE"], kw
    for kw in ({"N": -1}, {"H": 0}, {"H": 16385, "xs": 20000, "os": 20000}, {"xs": 63}, {"os": 63},
               {"r": FAKE, "rs": 63}, {"r": FAKE, "res": P(0x40000), "ress": 63}, {"r": FAKE, "res": OTHER},
               {"out": FAKE, "os": 72}, {"out": FAKE, "q": 1, "scale": FAKE}, {"r": P(0x50000), "rs": 72, "out": P(0x50000)},
               {"r": OTHER, "q": 1, "scale": FAKE}, {"r": P(0x50000), "res": FAKE, "ress": 72},
               {"r": P(0x50000), "res": P(0x50000), "ress": 72}):
        assert norm(lib, **kw) == S["TSA_ERR_SHAPE"], kw
    for kw in ({"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}):
        assert norm(lib, **kw) == S["TSA_ERR_VALUE"], kw
    for kw in ({"x": None}, {"w": None}, {"out": None}, {"q": 1}, {"res": P(0x40000)}):
        assert norm(lib, **kw) == S["TSA_ERR_NULL"], kw
    for kw in ({"x": ODD1}, {"w": ODD1}, {"wdt": 0, "w": ODD2}, {"r": ODD1}, {"out": ODD1}, {"r": FAKE, "res": ODD1},
               {"q": 1, "scale": ODD2}, {"rstd": ODD2}, {"dt": 0, "wdt": 0, "x": ODD2}):
        assert norm(lib, **kw) == S["TSA_ERR_ALIGN"], kw
    assert norm(lib, N=0, x=None, w=None, out=None) == S["TSA_OK"]


def test_quantize_rows_validation(lib):
    def q(x=FAKE, dt=2, N=2, H=64, xs=64, out=OTHER, os=64, scale=FAKE):
        return lib.tsa_quantize_rows(x, dt, N, H, xs, out, os, scale, None)

    assert q(dt=7) == S["TSA_ERR_DTYPE"]
    for kw in ({"N": -1}, {"H": 0}, {"H": 16385, "xs": 20000, "os": 20000}, {"xs": 63}, {"os": 63}, {"out": FAKE}):
        assert q(**kw) == S["TSA_ERR_SHAPE"], kw
    for kw in ({"x": None}, {"out": None}, {"scale": None}):
        assert q(**kw) == S["TSA_ERR_NULL"], kw
    for kw in ({"x": ODD1}, {"dt": 0, "x": ODD2}, {"scale": ODD2}):
        assert q(**kw) == S["TSA_ERR_ALIGN"], kw
    assert q(N=0, x=None, out=None, scale=None) == S["TSA_OK"]


def back(lib, g=FAKE, gs=64, x=FAKE, dt=2, N=2, H=64, xs=64, w=FAKE, wdt=2, rstd=FAKE, gr=None, grs=64, dx=OTHER,
         dxs=64, dw=OTHER, ws=FAKE, nws=1 << 30):
    return lib.tsa_rms_norm_backward(g, gs, x, dt, N, H, xs, w, wdt, rstd, gr, grs, dx, dxs, dw, ws, nws, None)


def test_rms_norm_backward_validation(lib):
    for kw in ({"dt": 3}, {"wdt": 1}):
        assert back(lib, **kw) == S["TSA_ERR_DTYPE"], kw
    for kw in ({"N": -1}, {"H": 0}, {"H": 16385, "xs": 20000, "gs": 20000, "dxs": 20000}, {"xs": 63}, {"gs": 63},
               {"dxs": 63}, {"gr": FAKE, "grs": 63}, {"dx": FAKE, "dxs": 72}, {"gr": OTHER, "grs": 72}):
        assert back(lib, **kw) == S["TSA_ERR_SHAPE"], kw
    for kw in ({"g": None}, {"x": None}, {"w": None}, {"rstd": None}, {"dx": None}, {"dw": None}):
        assert back(lib, **kw) == S["TSA_ERR_NULL"], kw
    for kw in ({"g": ODD1}, {"x": ODD1}, {"w": ODD1}, {"rstd": ODD2}, {"gr": ODD1}, {"dx": ODD1}, {"dw": ODD1},
               {"wdt": 0, "dw": ODD2}, {"ws": P(0x10010)}):
        assert back(lib, **kw) == S["TSA_ERR_ALIGN"], kw
    need = lib.tsa_rms_norm_backward_workspace_bytes(2, 64)
    assert need > 0 and lib.tsa_rms_norm_backward_workspace_bytes(0, 64) == 0
    # a part for each CTA at most, however many rows there are
    assert lib.tsa_rms_norm_backward_workspace_bytes(10**6, 64) == lib.tsa_rms_norm_backward_workspace_bytes(10**7, 64)
    assert back(lib, ws=None) == S["TSA_ERR_WORKSPACE"]
    assert back(lib, nws=need - 1) == S["TSA_ERR_WORKSPACE"]


def int8(lib, h=FAKE, M=2, H=64, hs=64, hsc=FAKE, w=FAKE, V=100, wst=64, wsc=FAKE, b=None, out=OTHER, dt=2, os=100,
         ws=FAKE, nws=1 << 20):
    return lib.tsa_lm_head_int8(h, M, H, hs, hsc, w, V, wst, wsc, b, out, dt, os, ws, nws, None)


def test_lm_head_int8_validation(lib):
    assert int8(lib, dt=3) == S["TSA_ERR_DTYPE"]
    for kw in ({"M": -1}, {"M": (1 << 20) + 1}, {"H": 8}, {"H": 24}, {"H": 16400, "hs": 16400, "wst": 16400}, {"V": 0}, {"hs": 48},
               {"wst": 48}, {"os": 99}):
        assert int8(lib, **kw) == S["TSA_ERR_SHAPE"], kw
    for kw in ({"h": None}, {"w": None}, {"hsc": None}, {"wsc": None}, {"out": None}):
        assert int8(lib, **kw) == S["TSA_ERR_NULL"], kw
    for kw in ({"h": ODD8}, {"w": ODD8}, {"hs": 72}, {"wst": 72}, {"hsc": ODD2}, {"wsc": ODD2}, {"b": ODD2},
               {"out": ODD1}, {"dt": 0, "out": ODD2}, {"ws": P(0x10010)}):
        assert int8(lib, **kw) == S["TSA_ERR_ALIGN"], kw
    need = lib.tsa_lm_head_int8_workspace_bytes(2, 64)
    assert need == 512 and lib.tsa_lm_head_int8_workspace_bytes(0, 64) == 0
    assert int8(lib, ws=None) == S["TSA_ERR_WORKSPACE"]
    assert int8(lib, nws=need - 1) == S["TSA_ERR_WORKSPACE"]
    assert int8(lib, M=0, h=None, w=None, out=None, ws=None) == S["TSA_OK"]


def xent(lib, h=FAKE, M=2, H=64, hs=64, w=FAKE, V=100, wst=64, b=None, cap=0.0, t=FAKE, rw=None, z=0.0, loss=FAKE,
         row=FAKE, lse=FAKE, dh=None, dhs=64, dw=None, dws=64, db=None, ws=FAKE, nws=1 << 40):
    return lib.tsa_lm_head_cross_entropy(h, M, H, hs, w, V, wst, b, cap, t, rw, z, loss, row, lse, dh, dhs, dw, dws, db,
                                         ws, nws, None)


def test_lm_head_cross_entropy_validation(lib):
    for kw in ({"M": -1}, {"M": (1 << 16) + 1}, {"H": 4}, {"H": 12}, {"H": 16392, "hs": 16392, "wst": 16392}, {"V": 0},
               {"hs": 32}, {"wst": 32}, {"dh": OTHER, "dhs": 32}, {"dw": OTHER, "dws": 32}, {"dh": FAKE}, {"dw": FAKE},
               {"b": OTHER, "db": OTHER}):
        assert xent(lib, **kw) == S["TSA_ERR_SHAPE"], kw
    for kw in ({"cap": -1.0}, {"cap": float("nan")}, {"cap": float("inf")}, {"z": float("nan")}, {"z": float("inf")}):
        assert xent(lib, **kw) == S["TSA_ERR_VALUE"], kw
    for kw in ({"h": None}, {"w": None}, {"t": None}, {"loss": None}, {"row": None}, {"lse": None}, {"db": OTHER}):
        assert xent(lib, **kw) == S["TSA_ERR_NULL"], kw
    for kw in ({"h": ODD8}, {"w": ODD8}, {"hs": 68}, {"wst": 68}, {"b": ODD2}, {"t": ODD4}, {"rw": ODD2}, {"loss": ODD2},
               {"row": ODD2}, {"lse": ODD2}, {"dh": ODD8}, {"dh": OTHER, "dhs": 68}, {"dw": ODD8},
               {"dw": OTHER, "dws": 68}, {"b": FAKE, "db": ODD2}, {"ws": P(0x10010)}):
        assert xent(lib, **kw) == S["TSA_ERR_ALIGN"], kw
    need = [lib.tsa_lm_head_cross_entropy_workspace_bytes(2, 64, 100, g, b) for g, b in ((0, 0), (1, 0), (1, 1))]
    assert 0 < need[0] < need[1] < need[2]
    assert lib.tsa_lm_head_cross_entropy_workspace_bytes(0, 64, 100, 1, 1) == 0
    for kw, n in (({}, need[0]), ({"dh": OTHER}, need[1]), ({"dw": OTHER}, need[1]), ({"b": FAKE, "db": OTHER}, need[2])):
        assert xent(lib, ws=None, **kw) == S["TSA_ERR_WORKSPACE"], kw
        assert xent(lib, nws=n - 1, **kw) == S["TSA_ERR_WORKSPACE"], kw


def test_calls_run_on_their_tensors_device(monkeypatch):
    import top_sampling_apply_gb300 as tsa
    from tests.test_abi_training import OnDevice1

    current, ran = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *a):
            current[0] = self.before

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return lambda *a: 256
            return lambda *a: ran.append((name, current[0])) or 0

    monkeypatch.setattr(tsa, "_lib", Lib())
    monkeypatch.setattr(tsa, "_current_device", lambda: current[0])
    monkeypatch.setattr(tsa, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(tsa, "_written", lambda tensors: None)
    monkeypatch.setattr(tsa.torch.cuda, "device", Device)
    monkeypatch.setattr(tsa.torch, "empty", OnDevice1)
    h, w = OnDevice1(2, 16, dtype=torch.bfloat16), OnDevice1(16, dtype=torch.bfloat16)
    q, f = OnDevice1(2, 16, dtype=torch.int8), OnDevice1(2)
    tsa.rms_norm(h, w, residual=h, quantize=True)
    tsa.rms_norm_backward(h, h, w, f, grad_residual=h)
    tsa.quantize_rows(h)
    tsa.lm_head_int8(q, f, q, f)
    tsa.lm_head_cross_entropy(h, h, OnDevice1(2, dtype=torch.int64), bias=f)
    assert ran == [("tsa_rms_norm", 1), ("tsa_rms_norm_backward", 1), ("tsa_quantize_rows", 1), ("tsa_lm_head_int8", 1),
                   ("tsa_lm_head_cross_entropy", 1)] and current == [0]


def test_binding_refuses_host_tensors():
    import top_sampling_apply_gb300 as tsa

    x, w = torch.zeros(2, 16), torch.zeros(16)
    b, q, v, i = x.bfloat16(), x.to(torch.int8), torch.zeros(2), torch.zeros(2, dtype=torch.int64)
    for call in (lambda: tsa.rms_norm(x, w), lambda: tsa.rms_norm_backward(x, x, w, v), lambda: tsa.quantize_rows(x),
                 lambda: tsa.lm_head_int8(q, v, q, v), lambda: tsa.lm_head_cross_entropy(b, b, i)):
        with pytest.raises(ValueError):
            call()


def test_refused_shapes_want_no_workspace(lib):
    """The binding makes room before the call checks its shapes: one that is refused must not ask for any."""
    x, q = lib.tsa_lm_head_cross_entropy_workspace_bytes, lib.tsa_lm_head_int8_workspace_bytes
    most = lib.tsa_max_vocab(2)
    for M, H, V in (((1 << 16) + 1, 64, 100), (1 << 40, 4096, 128256), (2, 16392, 100), (2, 1 << 50, 100),
                    (2, 64, most + 1), (2, 64, 1 << 60), (-1, 64, 100), (2, 0, 100), (2, 64, 0)):
        assert x(M, H, V, 1, 1) == 0, (M, H, V)
    for M, H in (((1 << 20) + 1, 64), (1 << 60, 64), (2, 16400), (2, 1 << 60), (0, 64), (2, 0)):
        assert q(M, H) == 0, (M, H)
    assert x(1 << 16, 16384, most, 1, 1) > 0 and q(1 << 20, 16384) == (1 << 20) * 16384 * 2
