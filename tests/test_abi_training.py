"""Host-side argument validation of the training-side calls (no GPU work): the documented status comes back
before anything is launched, and empty calls launch nothing."""
import ctypes

import pytest
import torch

from tests.test_abi import FAKE, S

ODD2, ODD4 = ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10004)


@pytest.fixture(scope="module")
def lib():
    from top_sampling_apply_gb300 import _build

    _build.build()
    import top_sampling_apply_gb300 as tsa

    return tsa.load_library()


def policy(lib, logits=FAKE, dtype=0, B=2, V=100, stride=100, mask=None, mstride=0, T=None, tok=FAKE, old=FAKE,
           adv=FAKE, ref=None, w=None, lo=0.2, hi=0.2, kl=0.0, ent=0.0, loss=FAKE, row=FAKE, lp=FAKE, entropy=None,
           grad=None, gstride=0, ws=None, nws=0):
    return lib.tsa_policy_loss(logits, dtype, B, V, stride, mask, mstride, T, 1.0, tok, old, adv, ref, w, lo, hi, kl,
                               ent, loss, row, lp, entropy, grad, gstride, ws, nws, None)


def test_policy_loss_validation(lib):
    for kw in ({"logits": None}, {"tok": None}, {"old": None}, {"adv": None}, {"loss": None}, {"row": None},
               {"lp": None}):
        assert policy(lib, **kw) == S["TSA_ERR_NULL"], kw
    for kw in ({"V": 0}, {"B": -1}, {"stride": 99}, {"grad": ctypes.c_void_p(0x20000), "gstride": 99},
               {"grad": FAKE, "gstride": 101}, {"V": lib.tsa_max_vocab(0) + 1, "stride": 10**7}):
        assert policy(lib, **kw) == S["TSA_ERR_SHAPE"], kw
    for kw in ({"lo": -0.1}, {"hi": -1.0}, {"lo": float("nan")}, {"hi": float("inf")}, {"kl": float("nan")},
               {"ent": float("inf")}):
        assert policy(lib, **kw) == S["TSA_ERR_VALUE"], kw
    assert policy(lib, dtype=3) == S["TSA_ERR_DTYPE"]
    assert policy(lib, mask=FAKE, mstride=3) == S["TSA_ERR_STRIDE"]
    for kw in ({"logits": ODD2}, {"tok": ODD4}, {"old": ODD2}, {"adv": ODD2}, {"ref": ODD2}, {"w": ODD2}, {"T": ODD2},
               {"loss": ODD2}, {"row": ODD2}, {"lp": ODD2}, {"entropy": ODD2}, {"grad": ODD2, "gstride": 100},
               {"mask": ODD2, "mstride": 4}):
        assert policy(lib, **kw) == S["TSA_ERR_ALIGN"], kw
    assert policy(lib, B=0, tok=None, old=None, adv=None, loss=None, row=None, lp=None) == S["TSA_OK"]


def test_policy_loss_workspace(lib):
    # rows of up to 512 KB are held on chip; longer ones keep 16 bytes a row between two passes
    for dt, most in ((0, 131072), (1, 262144), (2, 262144)):
        assert lib.tsa_policy_loss_workspace_bytes(7, most, dt) == 0
        assert lib.tsa_policy_loss_workspace_bytes(7, most + 64, dt) == 256
        assert lib.tsa_policy_loss_workspace_bytes(100, most + 64, dt) == 1792
    assert lib.tsa_policy_loss_workspace_bytes(0, 300000, 2) == 0
    long = dict(dtype=2, V=300000, stride=300000, grad=ctypes.c_void_p(0x20000), gstride=300000)
    assert policy(lib, **long) == S["TSA_ERR_WORKSPACE"]
    assert policy(lib, ws=FAKE, nws=255, **long) == S["TSA_ERR_WORKSPACE"]
    assert policy(lib, ws=ctypes.c_void_p(0x10010), nws=256, **long) == S["TSA_ERR_ALIGN"]


def preference(lib, logits=FAKE, N=4, V=100, stride=100, tok=FAKE, start=FAKE, P=1, w=None, ref=None, beta=0.1,
               smooth=0.0, margin=0.0, loss=FAKE, pair=FAKE, reward=FAKE, lp=FAKE, grad=None, gstride=0, ws=FAKE,
               nws=1 << 20, dtype=0):
    return lib.tsa_preference_loss(logits, dtype, N, V, stride, 1.0, tok, start, P, w, ref, beta, smooth, margin, 0,
                                   loss, pair, reward, lp, grad, gstride, ws, nws, None)


def test_preference_loss_validation(lib):
    for kw in ({"logits": None}, {"tok": None}, {"start": None}, {"loss": None}, {"pair": None}, {"reward": None},
               {"lp": None}):
        assert preference(lib, **kw) == S["TSA_ERR_NULL"], kw
    for kw in ({"V": 0}, {"N": -1}, {"P": -1}, {"stride": 99}, {"grad": FAKE, "gstride": 50}):
        assert preference(lib, **kw) == S["TSA_ERR_SHAPE"], kw
    for kw in ({"beta": float("nan")}, {"smooth": -0.1}, {"smooth": 1.1}, {"smooth": float("nan")},
               {"margin": float("inf")}):
        assert preference(lib, **kw) == S["TSA_ERR_VALUE"], kw
    assert preference(lib, dtype=9) == S["TSA_ERR_DTYPE"]
    for kw in ({"tok": ODD4}, {"start": ODD4}, {"w": ODD2}, {"ref": ODD2}, {"loss": ODD2}, {"pair": ODD2},
               {"reward": ODD2}, {"lp": ODD2}, {"ws": ctypes.c_void_p(0x10010)}):
        assert preference(lib, **kw) == S["TSA_ERR_ALIGN"], kw
    need = lib.tsa_preference_loss_workspace_bytes(4)
    assert need == 256 and lib.tsa_preference_loss_workspace_bytes(0) == 0
    assert preference(lib, ws=None) == S["TSA_ERR_WORKSPACE"]
    assert preference(lib, nws=need - 1) == S["TSA_ERR_WORKSPACE"]
    assert preference(lib, N=0, P=0, tok=None, start=None, loss=None, pair=None, reward=None, lp=None,
                      ws=None) == S["TSA_OK"]


def lm(lib, hidden=FAKE, M=2, H=64, hs=64, weight=FAKE, V=1000, wst=64, bias=None, cap=0.0, mask=None, mstride=0,
       T=None, tok=FAKE, out=FAKE, ws=FAKE, nws=1 << 30):
    return lib.tsa_lm_head_logprob(hidden, M, H, hs, weight, V, wst, bias, cap, mask, mstride, T, 1.0, tok, out, ws, nws,
                                   None)


def test_lm_head_logprob_validation(lib):
    for kw in ({"M": -1}, {"H": 4}, {"H": 12}, {"H": 16392, "hs": 16392, "wst": 16392}, {"V": 0}, {"hs": 32},
               {"wst": 32}):
        assert lm(lib, **kw) == S["TSA_ERR_SHAPE"], kw
    for kw in ({"cap": -1.0}, {"cap": float("nan")}, {"cap": float("inf")}):
        assert lm(lib, **kw) == S["TSA_ERR_VALUE"], kw
    for kw in ({"hidden": None}, {"weight": None}, {"tok": None}, {"out": None}):
        assert lm(lib, **kw) == S["TSA_ERR_NULL"], kw
    assert lm(lib, mask=FAKE, mstride=31) == S["TSA_ERR_STRIDE"]
    for kw in ({"hidden": ctypes.c_void_p(0x10008)}, {"weight": ctypes.c_void_p(0x10008)}, {"hs": 68}, {"wst": 68},
               {"bias": ODD2}, {"T": ODD2}, {"tok": ODD4}, {"out": ODD2}, {"ws": ctypes.c_void_p(0x10010)}):
        assert lm(lib, **kw) == S["TSA_ERR_ALIGN"], kw
    need = lib.tsa_lm_head_logprob_workspace_bytes(2, 1000)
    assert need > 0 and lib.tsa_lm_head_logprob_workspace_bytes(0, 1000) == 0
    # more rows than one pass takes share its workspace
    assert lib.tsa_lm_head_logprob_workspace_bytes(10**6, 1000) == lib.tsa_lm_head_logprob_workspace_bytes(8192, 1000)
    assert lm(lib, ws=None) == S["TSA_ERR_WORKSPACE"]
    assert lm(lib, nws=need - 1) == S["TSA_ERR_WORKSPACE"]
    assert lm(lib, M=0, hidden=None, weight=None) == S["TSA_OK"]


def table(**kw):
    import top_sampling_apply_gb300 as tsa

    t = (tsa._AdamTensor * 2)()
    for i in range(2):
        for f in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_exp", "exp_avg_sq_exp"):
            setattr(t[i], f, 0x10000)
        t[i].n = 10
    for f, v in kw.items():
        setattr(t[1], f, v)
    return t


def adam(lib, t=None, count=2, pd=0, gd=0, bits=32, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, step=1, scale=None):
    return lib.tsa_adamw_step(t, count, pd, gd, bits, lr, b1, b2, eps, wd, step, scale, 0, 0, None)


def test_adamw_validation(lib):
    t = table()
    for kw in ({"pd": 1}, {"pd": 3}, {"gd": 3}, {"gd": -1}):
        assert adam(lib, t, **kw) == S["TSA_ERR_DTYPE"], kw
    for kw in ({"bits": 16}, {"step": 0}, {"lr": -1.0}, {"lr": float("nan")}, {"b1": 1.0}, {"b1": -0.1}, {"b2": 1.0},
               {"b2": float("nan")}, {"eps": -1.0}, {"eps": float("inf")}, {"wd": -1.0}):
        assert adam(lib, t, **kw) == S["TSA_ERR_VALUE"], kw
    assert adam(lib, t, count=-1) == S["TSA_ERR_SHAPE"]
    assert adam(lib, None) == S["TSA_ERR_NULL"]
    assert adam(lib, table(n=-1)) == S["TSA_ERR_SHAPE"]
    assert adam(lib, table(n=(1 << 34) + 1)) == S["TSA_ERR_SHAPE"]
    for f in ("param", "grad", "exp_avg", "exp_avg_sq"):
        assert adam(lib, table(**{f: None})) == S["TSA_ERR_NULL"], f
        assert adam(lib, table(**{f: 0x10002})) == S["TSA_ERR_ALIGN"], f
    for f in ("exp_avg_exp", "exp_avg_sq_exp"):
        assert adam(lib, table(**{f: None}), bits=8) == S["TSA_ERR_NULL"], f
    assert adam(lib, t, scale=ODD2) == S["TSA_ERR_ALIGN"]
    # nothing to do: no launch
    assert adam(lib, None, count=0) == S["TSA_OK"]
    empty = table(n=0, param=None, grad=None)
    empty[0].n = 0
    assert adam(lib, empty) == S["TSA_OK"]


def test_adamw_state_values_validation(lib):
    out = (ctypes.c_void_p * 2)(0x10000, 0x10000)
    f = lib.tsa_adamw_state_values
    assert f(table(), 2, None, out, None) == S["TSA_ERR_NULL"]
    assert f(table(), 2, out, (ctypes.c_void_p * 2)(0x10000, None), None) == S["TSA_ERR_NULL"]
    assert f(table(), 2, (ctypes.c_void_p * 2)(0x10001, 0x10000), out, None) == S["TSA_ERR_ALIGN"]
    assert f(table(exp_avg_exp=None), 2, out, out, None) == S["TSA_ERR_NULL"]
    assert f(None, 0, None, None, None) == S["TSA_OK"]


def test_binding_rejects_host_tensors():
    import top_sampling_apply_gb300 as tsa

    x, i, v = torch.zeros(2, 10), torch.zeros(2, dtype=torch.int64), torch.zeros(2)
    with pytest.raises(ValueError):
        tsa.policy_loss(x, i, v, v)
    with pytest.raises(ValueError):
        tsa.preference_loss(x, i, torch.tensor([0, 1, 2]))
    h = torch.zeros(2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tsa.lm_head_logprob(h, h, i)
    with pytest.raises(ValueError):
        tsa.adamw_plan([v], [v], [v], [v])
    with pytest.raises(ValueError):
        tsa.adamw_state([v], 16)


class OnDevice1:
    """What the binding asks of a tensor, for one on cuda:1."""
    is_cuda, device, requires_grad, _base = True, torch.device("cuda", 1), False, None

    def __init__(self, *shape, dtype=torch.float32, **kw):
        shape = shape[0] if shape and isinstance(shape[0], tuple) else shape
        self.shape, self.dtype = torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def size(self, i):
        return self.shape[i]

    def numel(self):
        return self.shape.numel()

    def stride(self, i):
        return self.shape[i + 1:].numel()

    def get_device(self):
        return 1

    def is_contiguous(self):
        return True

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 0x10000

    def untyped_storage(self):
        return self


def test_calls_run_on_their_tensors_device(monkeypatch):
    # a launch goes to the current device: each call makes its tensors' device current, and leaves things as they were
    import top_sampling_apply_gb300 as tsa

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
                return lambda *a: 0
            return lambda *a: ran.append((name, current[0])) or 0

    monkeypatch.setattr(tsa, "_lib", Lib())
    monkeypatch.setattr(tsa, "_current_device", lambda: current[0])
    monkeypatch.setattr(tsa, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(tsa, "_stream", lambda t: 0)
    monkeypatch.setattr(tsa, "_written", lambda tensors: None)
    monkeypatch.setattr(tsa.torch.cuda, "device", Device)
    monkeypatch.setattr(tsa.torch, "empty", OnDevice1)
    f, i, h = OnDevice1(2), OnDevice1(2, dtype=torch.int64), OnDevice1(2, 16, dtype=torch.bfloat16)
    x, bits = OnDevice1(2, 32), OnDevice1(2, 1, dtype=torch.int32)
    tsa.policy_loss(x, i, f, f)
    tsa.preference_loss(x, i, OnDevice1(3, dtype=torch.int64))
    tsa.lm_head_logprob(h, h, i)
    tsa.adamw_step(tsa.adamw_plan([f], [f], [f], [f]), 1, 0.1)
    tsa.sample(x)
    tsa.sample_icdf(x, f)
    tsa.sample_noalloc(x, i)
    tsa.topk(x, 2)
    tsa.selective_log_softmax(x, i)
    tsa.apply_token_bitmask(x, bits)
    tsa.lm_head_topk(h, h, 2)
    tsa.bitmask_from_allowed(OnDevice1(2, 32, dtype=torch.bool))
    assert [n for n, d in ran if d != 1] == [] and len(ran) == 12 and current == [0]
    ran.clear()
    current[0] = 1  # already current
    monkeypatch.setattr(tsa.torch.cuda, "device", None)
    tsa.policy_loss(x, i, f, f)
    assert ran == [("tsa_policy_loss", 1)]


def test_an_error_leaves_the_device_as_it_was(monkeypatch):
    import top_sampling_apply_gb300 as tsa

    left = []

    class Device:
        def __init__(self, index):
            pass

        def __enter__(self):
            pass

        def __exit__(self, *a):
            left.append(1)

    tsa.load_library()
    monkeypatch.setattr(tsa, "_current_device", lambda: 0)
    monkeypatch.setattr(tsa.torch.cuda, "device", Device)
    with pytest.raises(tsa.TSAError) as e:
        tsa._call(1, lambda *a: S["TSA_ERR_SHAPE"], 1, 2)
    assert left == [1] and e.value.status == S["TSA_ERR_SHAPE"]


def test_a_plan_checks_its_tensors_however_it_is_made():
    import top_sampling_apply_gb300 as tsa

    v = torch.zeros(2)
    with pytest.raises(ValueError):
        tsa.AdamWPlan([v], [v], [v], [v])
    with pytest.raises(ValueError):
        tsa.AdamWPlan([v], [], [v], [v])
    with pytest.raises(ValueError):
        tsa.AdamWPlan([], [], [], [], [v], [v])


def test_what_is_set_on_kernels_is_kept_for_any_number_of_them(tmp_path):
    # kernels times devices may pass any fixed count: one process on eight GPUs has hundreds
    import os
    import subprocess

    src = tmp_path / "table.cpp"
    src.write_text(r"""
#include "tsa_prepared.h"
#include <cstdio>
int main() {
    static tsa::PreparedTable t;
    static char fn[300];
    tsa::Prepared *at[300][8];
    for (int i = 0; i < 300; ++i)
        for (int d = 0; d < 8; ++d) {
            tsa::Prepared *p = t.find(fn + i, d);
            if (!p || p->smem != 0 || p->cluster16 != 0) return 1;
            p->smem = 1000 * i + d;
            at[i][d] = p;
        }
    for (int i = 0; i < 300; ++i)
        for (int d = 0; d < 8; ++d) {
            tsa::Prepared *p = t.find(fn + i, d);
            if (p != at[i][d] || p->fn != fn + i || p->device != d || p->smem != (size_t)(1000 * i + d)) return 2;
        }
    return 0;
}
""")
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_sampling_apply_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", csrc, str(src), "-o", str(tmp_path / "table")], check=True)
    assert subprocess.run([str(tmp_path / "table")]).returncode == 0


def test_no_gradient_asked_for(monkeypatch):
    # None, like False, asks for the loss alone: there is nothing to raise the version of
    import top_sampling_apply_gb300 as tsa

    class Lib:
        def __getattr__(self, name):
            return (lambda *a: 256) if name.endswith("_bytes") else lambda *a: 0

    monkeypatch.setattr(tsa, "_lib", Lib())
    monkeypatch.setattr(tsa, "_current_device", lambda: 1)
    monkeypatch.setattr(tsa, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(tsa.torch, "empty", OnDevice1)
    f, i, x = OnDevice1(2), OnDevice1(2, dtype=torch.int64), OnDevice1(2, 32)
    for grad in (None, False):
        assert tsa.policy_loss(x, i, f, f, grad=grad).grad is None
        assert tsa.preference_loss(x, i, OnDevice1(3, dtype=torch.int64), grad=grad).grad is None
