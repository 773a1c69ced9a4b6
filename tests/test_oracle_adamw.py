"""Pins of the float64 AdamW step and of its 8-bit grids."""
import numpy as np
import pytest
import torch

from oracle import adamw


def test_step_against_torch_in_float64():
    rng = np.random.default_rng(0)
    p0 = rng.standard_normal(50)
    p = torch.nn.Parameter(torch.from_numpy(p0.copy()))
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.8, 0.95), eps=1e-7, weight_decay=0.2, foreach=False)
    q, m, v = p0, np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.from_numpy(g)
        opt.step()
        q, m, v = adamw.step(q, g, m, v, t, 3e-3, 0.8, 0.95, 1e-7, 0.2)
    assert np.allclose(p.detach().numpy(), q, rtol=1e-13, atol=1e-15)


def test_codes_are_upper_halves_of_floats():
    # the definition in bits: code c of base b is the float with bits (c + 8 b) << 20
    for b in (0, 1, 97, 200):
        c = np.arange(256)
        bits = np.where(c > 0, (c + 8 * b) << 20, 0).astype(np.uint32)
        want = bits.view(np.float32).astype(np.float64)
        assert np.array_equal(adamw.value(c, np.array([b]), False), want)
    signed = adamw.value(np.array([5, 133]), np.array([100]), True)
    assert signed[0] > 0 and signed[1] == -signed[0]


@pytest.mark.parametrize("signed", [False, True])
def test_grid_values_round_to_themselves_and_within_a_step(signed):
    rng = np.random.default_rng(1)
    x = np.exp(rng.uniform(-12, 0, 256)) * (np.sign(rng.standard_normal(256)) if signed else 1)
    exps = adamw.base(x, 14 if signed else 30)
    r = rng.integers(0, 65536, 256)
    y = adamw.grid(x, exps, signed, r)
    assert np.array_equal(adamw.grid(y, exps, signed, r * 0), y)
    big = np.abs(x) > np.abs(x).max() * 2.0 ** -12
    assert np.all(np.abs(y - x)[big] <= np.abs(x)[big] * (1 / 16 if signed else 1 / 8))
    # y is one of the codes
    codes = adamw.value(np.arange(256), np.repeat(exps[:1], 1), signed)
    assert np.all(np.isin(y, codes))


def test_stochastic_rounding_has_the_right_mean_and_keeps_small_values():
    x = np.concatenate([[1.0], np.full(255, 0.3)])
    exps = adamw.base(x, 30)
    mean = np.mean([adamw.grid(x, exps, False, np.full(256, r))[1] for r in range(0, 65536, 64)])
    assert mean == pytest.approx(0.3, rel=1e-3)
    tiny = np.concatenate([[1.0], np.full(255, 1e-30)])
    assert np.all(adamw.grid(tiny, adamw.base(tiny, 30), False, np.zeros(256)) > 0)


def test_bf16_by_word_brackets():
    p = np.array([1.003, -2.7, 0.0, 1e-5])
    lo = adamw.bf16_by_word(p, np.zeros(4, np.uint64))
    hi = adamw.bf16_by_word(p, np.full(4, 0xFFFFFFFF, np.uint64))
    assert np.all(np.abs(lo) <= np.abs(p)) and np.all(np.abs(hi) >= np.abs(p))
    t = torch.from_numpy(np.stack([lo, hi]))
    assert torch.equal(t.to(torch.bfloat16).double(), t)
