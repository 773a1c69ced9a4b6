"""The AdamW step on the GPU against its float64 definition.

Tolerances, u = 2^-24: m' and v' are two products and a sum (the square one product more) on a scaled
gradient, so they are off by at most 4 u (|beta1 m| + |(1 - beta1) g|) and 6 u v'.  The update is a quotient of
these through an approximate square root (2^-22) and division (2^-21): 2^-20 of itself plus m's absolute error
over the denominator; then p takes two roundings, and one to bf16 by the element's random word.  A code must
be one that the exact value moved by the tolerance rounds to."""
import numpy as np
import pytest
import torch

from oracle import adamw

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def tsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import top_sampling_apply_gb300 as lib

    lib.load_library()
    return lib


def make(rng, sizes, pdt, gdt, bits, shift=0):
    """Tensors of the sizes, each `shift` elements into its own guarded buffer."""
    out = []
    for n in sizes:
        t = {"n": n}
        size = np.exp(rng.standard_normal((n + 255) // 256 or 1)).repeat(256)[:n]

        def put(a, dt, shift=shift):
            buf = torch.zeros(len(a) + 64, dtype=dt, device=DEV)
            buf[:] = 77 if dt == torch.uint8 else 7.0
            view = buf[shift:shift + len(a)]
            view.copy_(torch.from_numpy(np.asarray(a)).to(DEV))
            return buf, view

        t["p"] = put((0.1 * rng.standard_normal(n)).astype(np.float32), pdt)
        t["g"] = put((1e-2 * size * rng.standard_normal(n)).astype(np.float32), gdt)
        if bits == 32:
            t["m"] = put((1e-3 * size * rng.standard_normal(n)).astype(np.float32), torch.float32)
            t["v"] = put(((1e-2 * size) ** 2 * rng.random(n)).astype(np.float32), torch.float32)
        else:
            t["m"] = put(rng.integers(0, 256, n).astype(np.uint8), torch.uint8)
            t["v"] = put(rng.integers(0, 256, n).astype(np.uint8), torch.uint8)
            blocks = (n + 255) // 256
            t["me"] = put(rng.integers(98, 104, blocks).astype(np.uint8), torch.uint8, 0)
            t["ve"] = put(rng.integers(76, 84, blocks).astype(np.uint8), torch.uint8, 0)
        out.append(t)
    return out


def plan_of(tsa, ts, bits):
    pick = lambda k: [t[k][1] for t in ts]  # noqa: E731
    if bits == 32:
        return tsa.adamw_plan(pick("p"), pick("g"), pick("m"), pick("v"))
    return tsa.adamw_plan(pick("p"), pick("g"), pick("m"), pick("v"), pick("me"), pick("ve"))


def arr(x):
    return x.cpu().to(torch.float64).numpy() if x.dtype != torch.uint8 else x.cpu().numpy().astype(np.int64)


def values(t, bits):
    if bits == 32:
        return arr(t["m"][1]), arr(t["v"][1])
    return (adamw.value(arr(t["m"][1]), arr(t["me"][1]), True), adamw.value(arr(t["v"][1]), arr(t["ve"][1]), False))


def check_step(ts, before, k0, bits, pdt, t, scale, seed, offset, hp=HP):
    for k, (x, old) in enumerate(zip(ts, before)):
        n = x["n"]
        if n == 0:
            continue
        p, g, m, v = old
        pe, me, ve = adamw.step(p, g, m, v, t, hp["lr"], hp["beta1"], hp["beta2"], hp["eps"], hp["weight_decay"],
                                scale)
        tm = 4 * U * (np.abs(hp["beta1"] * m) + np.abs((1 - hp["beta1"]) * g * scale)) + 1e-45
        tv = 6 * U * ve + 1e-45
        mg, vg = values(x, bits)
        word = adamw.words(seed, offset, k0 + k, n)
        if bits == 32:
            assert np.all(np.abs(mg - me) <= tm) and np.all(np.abs(vg - ve) <= tv)
        else:
            r = (word & np.uint64(0xFFFF)).astype(np.float64)
            eb, vb = arr(x["me"][1]), arr(x["ve"][1])
            for b, ref, tol, span in ((eb, me, tm, 14), (vb, ve, tv, 30)):
                assert np.all((b >= adamw.base(np.maximum(np.abs(ref) - tol, 0), span)) &
                              (b <= adamw.base(np.abs(ref) + tol, span)))
            for got, ref, tol, b, signed in ((mg, me, tm, eb, True), (vg, ve, tv, vb, False)):
                lo, hi = (adamw.grid(ref + s * tol, b, signed, r) for s in (-1, 1))
                assert np.all((got >= lo) & (got <= hi))
        c1, c2 = 1 - hp["beta1"] ** t, 1 - hp["beta2"] ** t
        den = np.sqrt(ve / c2) + hp["eps"]
        upd = hp["lr"] / c1 * np.abs(me) / den
        tp = upd * 2.0 ** -20 + hp["lr"] / c1 * tm / den + 3 * U * np.abs(pe) + 1e-45
        pg = arr(x["p"][1])
        if pdt == torch.float32:
            assert np.all(np.abs(pg - pe) <= tp)
        else:
            lo, hi = adamw.bf16_by_word(pe - tp, word), adamw.bf16_by_word(pe + tp, word)
            assert np.all((pg >= lo) & (pg <= hi))


def check_guards(ts, shift):
    for t in ts:
        for key, (buf, view) in ((k, t[k]) for k in t if k != "n"):
            s = 0 if key in ("me", "ve") else shift
            rest = torch.cat([buf[:s], buf[s + view.numel():]])
            assert torch.all(rest == (77 if buf.dtype == torch.uint8 else 7.0)), key


SIZES = [1, 7, 0, 255, 256, 257, 5000, 8, 70001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gdt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 3])
def test_steps(tsa, bits, pdt, gdt, shift):
    ts = make(np.random.default_rng(1), SIZES, pdt, gdt, bits, shift)
    plan = plan_of(tsa, ts, bits)
    scale = torch.full((1,), 0.375, device=DEV)
    for t in (1, 2, 3):
        before = [(arr(x["p"][1]), arr(x["g"][1]), *values(x, bits)) for x in ts]
        tsa.adamw_step(plan, t, grad_scale=scale, seed=2 ** 40 + 5, offset=t, **HP)
        check_step(ts, before, 0, bits, pdt, t, 0.375, 2 ** 40 + 5, t)
    check_guards(ts, shift)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(tsa, bits):
    # more tensors than one launch's table; the random row is the tensor's place in the list
    rng = np.random.default_rng(2)
    ts = make(rng, rng.integers(0, 900, 1100).tolist(), torch.bfloat16, torch.bfloat16, bits)
    before = [(arr(x["p"][1]), arr(x["g"][1]), *values(x, bits)) for x in ts]
    tsa.adamw_step(plan_of(tsa, ts, bits), 7, seed=9, offset=7, **HP)
    check_step(ts, before, 0, bits, torch.bfloat16, 7, 1.0, 9, 7)
    check_guards(ts, 0)


def test_large_tensor_with_chunks(tsa):
    n = 20_000_003
    g = torch.Generator(device=DEV).manual_seed(1)
    p = torch.randn(n, generator=g, device=DEV).to(torch.bfloat16)
    grad = torch.randn(n, generator=g, device=DEV).mul_(1e-2).to(torch.bfloat16)
    m, v, me, ve = tsa.adamw_state([p], 8)
    plan = tsa.adamw_plan([p], [grad], m, v, me, ve)
    tsa.adamw_step(plan, 1, 1e-3, weight_decay=0.0)
    wm, wv = tsa.adamw_state_values(plan)
    # from zero states m' = (1 - b1) g and v' = (1 - b2) g^2: a sixteenth and an eighth of relative error
    e = grad.float() * 0.1
    big = e.abs() > 1e-5
    assert ((wm[0].float() - e).abs() <= e.abs() / 15.9)[big].all()
    s = grad.float().square() * 1e-3
    big = s > 1e-12
    assert ((wv[0].float() - s).abs() <= s / 7.9)[big].all()
    # the stochastic rounding of v' is unbiased: 2e7 roundings with errors under 1/8 of independent signs
    assert abs((wv[0].double().sum() / s.double().sum()).item() - 1) < 2e-4


def test_state_values(tsa):
    for shift in (0, 3):
        ts = make(np.random.default_rng(3), SIZES, torch.bfloat16, torch.float32, 8, shift)
        plan = plan_of(tsa, ts, 8)
        m, v = tsa.adamw_state_values(plan)
        for x, a, b in zip(ts, m, v):
            wm, wv = values(x, 8)
            assert np.array_equal(arr(a), wm) and np.array_equal(arr(b), wv)


def test_nonfinite_scale_changes_nothing_and_equal_steps_equal_bits(tsa):
    a = make(np.random.default_rng(4), [3000], torch.bfloat16, torch.bfloat16, 8)
    b = make(np.random.default_rng(4), [3000], torch.bfloat16, torch.bfloat16, 8)
    for bad in (float("inf"), float("nan")):
        tsa.adamw_step(plan_of(tsa, a, 8), 1, grad_scale=torch.full((1,), bad, device=DEV), **HP)
    for k in ("p", "m", "v", "me", "ve"):
        assert torch.equal(a[0][k][1], b[0][k][1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tsa.adamw_step(plan_of(tsa, a, 8), 1, seed=3, offset=1, **HP)
    with torch.cuda.stream(side):
        tsa.adamw_step(plan_of(tsa, b, 8), 1, seed=3, offset=1, **HP)
    torch.cuda.synchronize()
    for k in ("p", "m", "v", "me", "ve"):
        assert torch.equal(a[0][k][1], b[0][k][1])


@pytest.mark.parametrize("bits", [32, 8])
def test_nonfinite_gradients_stay_local(tsa, bits):
    a = make(np.random.default_rng(5), [600], torch.float32, torch.float32, bits)
    b = make(np.random.default_rng(5), [600], torch.float32, torch.float32, bits)
    a[0]["g"][1][10] = float("nan")
    a[0]["g"][1][300] = float("inf")
    b[0]["g"][1][10] = 0.0
    b[0]["g"][1][300] = 0.0
    for t in (a, b):
        tsa.adamw_step(plan_of(tsa, t, bits), 5, **HP)
    p, q = a[0]["p"][1], b[0]["p"][1]
    assert torch.isnan(p[10]) and not torch.isfinite(p[300])
    rest = torch.ones(600, dtype=torch.bool, device=DEV)
    rest[10] = rest[300] = False
    assert torch.equal(p[rest], q[rest])


def test_zero_gradients_keep_zero_states_and_decay(tsa):
    p = torch.full((1000,), 2.0, device=DEV)
    g = torch.zeros(1000, device=DEV)
    for bits in (32, 8):
        st = tsa.adamw_state([p], bits)
        q = p.clone()
        tsa.adamw_step(tsa.adamw_plan([q], [g], *st), 1, 0.1, weight_decay=0.5)
        assert torch.all(q == 1.9) and all(torch.all(s == 0) for lst in st if lst for s in lst)


def test_second_moment_reaches_its_mean(tsa):
    # with beta2 = 0.99 a constant |g| must bring v to g^2: rounding to nearest would stop far below
    n = 256 * 64
    p = torch.zeros(n, device=DEV, dtype=torch.bfloat16)
    g = torch.full((n,), 0.5, device=DEV)
    plan = tsa.adamw_plan([p], [g], *tsa.adamw_state([p], 8))
    for t in range(1, 801):
        tsa.adamw_step(plan, t, 0.0, beta2=0.99, seed=1, offset=t)
    v = tsa.adamw_state_values(plan)[1][0].float().mean().item()
    # 1 - 0.99^800 is 0.9997; a rounding error of at most 1/8 a step, decaying with 0.99, over 16384 elements
    assert abs(v / 0.25 - 1) < 0.02


def test_refusals(tsa):
    p, g = torch.zeros(4, device=DEV), torch.zeros(4, device=DEV)
    m, v, _, _ = tsa.adamw_state([p], 32)
    for bad in (dict(params=[p.half()]), dict(params=[p.cpu()]), dict(grads=[g[:3]]), dict(grads=[]),
                dict(exp_avg=[m[0].double()]), dict(exp_avg_sq=[v[0][::2]]), dict(exp_avg_exp=[m[0]])):
        a = dict(params=[p], grads=[g], exp_avg=m, exp_avg_sq=v)
        a.update(bad)
        with pytest.raises(ValueError):
            tsa.adamw_plan(**a)
    c8 = tsa.adamw_state([p], 8)
    with pytest.raises(ValueError):
        tsa.adamw_plan([p], [g], c8[0], c8[1])
    plan = tsa.adamw_plan([p], [g], m, v)
    for kw in (dict(step=0), dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1),
               dict(eps=float("inf")), dict(weight_decay=-0.1)):
        with pytest.raises(tsa.TSAError):
            tsa.adamw_step(plan, **{**dict(step=1, lr=0.1), **kw})
    with pytest.raises(ValueError):
        tsa.adamw_step(plan, 1, 0.1, grad_scale=torch.ones(1))
    with pytest.raises(ValueError):
        tsa.adamw_state_values(plan)
    tsa.adamw_step(tsa.adamw_plan([], [], [], []), 1, 0.1)  # an empty list is a no-op


@pytest.mark.parametrize("pdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("eps", [0.0, 1e-25])
def test_second_moments_below_the_normal_numbers(tsa, pdt, eps):
    # gradients of 1e-20 to 1e-17: v' is 1e-43 to 1e-37, and with no eps to speak of the step still has the size of lr.
    # v' is a square, a product and a sum with an absolute error of 2^-150 each beside their relative ones, and its
    # root has half its relative error.
    rng = np.random.default_rng(6)
    n = 3001
    p = torch.from_numpy((0.1 * rng.standard_normal(n)).astype(np.float32)).to(DEV).to(pdt)
    g = torch.from_numpy((10.0 ** rng.uniform(-20, -17, n) * rng.choice([-1, 1], n)).astype(np.float32)).to(DEV)
    m, v, _, _ = tsa.adamw_state([p], 32)
    old = arr(p)
    pe, me, ve = adamw.step(old, arr(g), np.zeros(n), np.zeros(n), 1, 1e-2, 0.9, 0.999, eps, 0.0)
    tsa.adamw_step(tsa.adamw_plan([p], [g], m, v), 1, 1e-2, eps=eps, weight_decay=0.0, seed=8, offset=1)
    upd = np.abs(pe - old)
    assert upd.min() > 5e-3
    tv = 6 * U * ve + 3 * 2.0 ** -150
    assert np.all(np.abs(arr(v[0]) - ve) <= tv)
    tp = upd * (2.0 ** -20 + 4 * U + tv / ve) + 3 * U * np.abs(pe)
    if pdt == torch.float32:
        assert np.all(np.abs(arr(p) - pe) <= tp)
    else:
        word = adamw.words(8, 1, 0, n)
        assert np.all((arr(p) >= adamw.bf16_by_word(pe - tp, word)) & (arr(p) <= adamw.bf16_by_word(pe + tp, word)))


def test_a_step_is_seen_by_autograd(tsa):
    p = torch.randn(8, device=DEV, requires_grad=True)
    flat = torch.randn(12, device=DEV)
    q, r = flat[:5], flat[5:]
    x = torch.randn(5, device=DEV, requires_grad=True)
    y, z = (p * p).sum(), (x * q).sum()  # their backward needs p and q as they were
    ps = [p, q, r]
    plan = tsa.adamw_plan(ps, [torch.ones_like(t) for t in ps], *tsa.adamw_state(ps, 8))
    tsa.adamw_step(plan, 1, 0.1)
    for loss in (y, z):
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    (p * p).sum().backward()
    outs = [[torch.empty(t.shape, dtype=torch.bfloat16, device=DEV) for t in ps] for _ in range(2)]
    versions = [t._version for o in outs for t in o]
    tsa.adamw_state_values(plan, *outs)
    assert all(t._version > v for t, v in zip(outs[0] + outs[1], versions))
    with torch.inference_mode():
        t = torch.ones(4, device=DEV)
    tsa.adamw_step(tsa.adamw_plan([t], [torch.ones(4, device=DEV)], *tsa.adamw_state([t], 32)), 1, 0.1)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_plan_keeps_the_memory_it_writes(tsa, bits):
    # a parameter that moves to other memory, and states that are dropped: what is allocated next is not the plan's
    n = 3 << 20
    p, g = torch.zeros(n, device=DEV), torch.ones(n, device=DEV)
    st = tsa.adamw_state([p], bits)
    plan = tsa.adamw_plan([p], [g], *st)
    where = [p.data_ptr(), st[0][0].data_ptr(), st[1][0].data_ptr()]
    p.data = torch.full((n,), 2.0, device=DEV)
    for t in st[0] + st[1]:
        t.data = torch.empty(0, device=DEV, dtype=t.dtype)
    new = [torch.full((n,), 7, device=DEV, dtype=dt) for dt in 2 * [torch.float32, st[0][0].dtype, st[1][0].dtype]]
    assert not {t.data_ptr() for t in new} & set(where)
    tsa.adamw_step(plan, 1, 0.1)
    assert all(torch.all(t == 7) for t in new) and torch.all(p == 2.0)


@pytest.mark.parametrize("bits", [32, 8])
def test_replays_in_a_graph(tsa, bits):
    keys = ("p", "g", "m", "v") + (("me", "ve") if bits == 8 else ())
    a, b, w = (make(np.random.default_rng(8), [3000, 17], torch.bfloat16, torch.bfloat16, bits) for _ in range(3))
    scale = torch.full((1,), 0.5, device=DEV)

    def step(plan):
        tsa.adamw_step(plan, 4, grad_scale=scale, seed=11, offset=4, **HP)

    step(plan_of(tsa, w, bits))
    if bits == 8:
        tsa.adamw_state_values(plan_of(tsa, w, bits))
    torch.cuda.synchronize()
    plan = plan_of(tsa, a, bits)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(plan)
        vals = tsa.adamw_state_values(plan) if bits == 8 else None
    eager = plan_of(tsa, b, bits)
    for k in range(2):
        for t in a + b:
            t["g"][1].copy_(torch.arange(t["n"], device=DEV) * (1e-4 * (k + 1)))
        g.replay()
        step(eager)
        for x, y in zip(a, b):
            for key in keys:
                assert torch.equal(x[key][1], y[key][1]), key
        if bits == 8:
            for x, y in zip(vals, tsa.adamw_state_values(eager)):
                assert all(torch.equal(p, q) for p, q in zip(x, y))


@pytest.mark.parametrize("bits", [32, 8])
def test_several_tables_of_tensors_of_several_chunks(tsa, bits):
    # 600 tensors are two tables, and three million elements make a chunk 2,048 of them
    rng = np.random.default_rng(7)
    ts = make(rng, rng.integers(1, 10001, 600).tolist(), torch.bfloat16, torch.bfloat16, bits)
    assert sum(t["n"] for t in ts) > 152 * 16 * 1024
    before = [(arr(x["p"][1]), arr(x["g"][1]), *values(x, bits)) for x in ts]
    tsa.adamw_step(plan_of(tsa, ts, bits), 3, seed=10, offset=3, **HP)
    check_step(ts, before, 0, bits, torch.bfloat16, 3, 1.0, 10, 3)
    check_guards(ts, 0)
