"""Pins of the float64 forms around the vocabulary head: gradients against central differences, closed forms,
and torch's own float64 functions."""
import pytest
import torch

from oracle import head


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def difference(f, x, d, step=1e-5):
    return (f(x + step * d) - f(x - step * d)) / (2 * step)


@pytest.mark.parametrize("cap,z_loss,bias,weighted", [(0.0, 0.0, False, False), (3.0, 0.0, True, True),
                                                       (0.0, 0.01, True, False), (2.0, 0.1, False, True)])
def test_cross_entropy_gradients_against_differences(cap, z_loss, bias, weighted):
    M, V, H = 5, 11, 7
    h, w = rand(M, H, seed=1), rand(V, H, seed=2)
    b = rand(V, seed=3) if bias else None
    t = torch.tensor([0, 10, -1, 4, 4])
    rw = torch.tensor([0.5, 0.0, 1.0, -2.0, 0.25], dtype=torch.float64) if weighted else None
    r = head.cross_entropy(h, w, t, b, cap, rw, z_loss)
    for name, x, f in (("dh", h, lambda x: head.cross_entropy(x, w, t, b, cap, rw, z_loss)["loss"]),
                       ("dw", w, lambda x: head.cross_entropy(h, x, t, b, cap, rw, z_loss)["loss"])):
        for seed in range(4):
            d = rand(*x.shape, seed=seed + 9)
            assert abs(difference(f, x, d) - (r[name] * d).sum()) < 1e-8
    if bias:
        d = rand(V, seed=7)
        f = lambda x: head.cross_entropy(h, w, t, x, cap, rw, z_loss)["loss"]  # noqa: E731
        assert abs(difference(f, b, d) - (r["db"] * d).sum()) < 1e-8
    assert (r["dh"][2] == 0).all() and r["row"][2] == 0
    if weighted:
        assert (r["dh"][1] == 0).all()


def test_cross_entropy_is_torchs():
    h, w, t = rand(6, 5, seed=1), rand(9, 5, seed=2), torch.tensor([0, 8, -100, 3, 3, -100])
    r = head.cross_entropy(h, w, t)
    want = torch.nn.functional.cross_entropy(h @ w.T, t, ignore_index=-100)
    assert abs(r["loss"] - want) < 1e-14
    assert torch.allclose(r["lse"][0], torch.logsumexp(h[0] @ w.T, -1))


@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.1])
def test_norm_gradients_against_differences(eps):
    x, w, g = rand(4, 9, seed=1), rand(9, seed=2), rand(4, 9, seed=3)
    gr = rand(4, 9, seed=4)
    rstd = head.rms_norm(x, w, eps)[1]
    dx, dw = head.rms_norm_backward(g, x, w, rstd, gr)[:2]
    for seed in range(4):
        d = rand(4, 9, seed=seed + 20)
        f = lambda y: (head.rms_norm(y, w, eps)[0] * g).sum() + (y * gr).sum()  # noqa: E731
        assert abs(difference(f, x, d) - (dx * d).sum()) < 1e-8
        d = rand(9, seed=seed + 30)
        f = lambda v: (head.rms_norm(x, v, eps)[0] * g).sum()  # noqa: E731
        assert abs(difference(f, w, d) - (dw * d).sum()) < 1e-8


def test_norm_closed_forms():
    y, rstd = head.rms_norm(torch.tensor([[3.0, 4.0]]), torch.tensor([1.0, 2.0]), 0.0)
    k = 1 / 12.5 ** 0.5
    assert torch.allclose(y, torch.tensor([[3 * k, 8 * k]], dtype=torch.float64)) and abs(rstd - k) < 1e-15
    q, scale = head.quantize(torch.tensor([[-254.0, 127.0, 1.0], [0.0, 0.0, 0.0]]))
    assert scale.tolist() == [2.0, 0.0] and q.tolist() == [[-127.0, 63.5, 0.5], [0.0, 0.0, 0.0]]


def test_int8_scores():
    h, w = torch.tensor([[1, -2]], dtype=torch.int8), torch.tensor([[3, 4], [-128, 127]], dtype=torch.int8)
    s, z = head.int8_scores(h, torch.tensor([0.5]), w, torch.tensor([2.0, 1.0]), torch.tensor([0.0, 1.0]))
    assert s.tolist() == [[-5.0, -382.0]] and z.tolist() == [[-5.0, -190.0]]
