"""The calls around the vocabulary head in float64, from their formulas: the root-mean-square norm with its
8-bit rows and its gradients, the scores of an 8-bit head, and the cross entropy of the head's scores with its
gradients.  Plain torch on whatever device the inputs are on."""
import torch


def add_residual(x, r):
    """The sum as the rows' type holds it."""
    return x if r is None else (x.double() + r.double()).to(x.dtype)


def rms_norm(s, w, eps):
    """(y, 1 / rms) of rows s, unrounded."""
    s = s.double()
    rstd = 1.0 / torch.sqrt((s * s).mean(-1) + eps)
    return s * rstd[:, None] * w.double(), rstd


def rms_norm_backward(g, s, w, rstd, gr=None):
    """(dx, dw, and the sums of absolute terms that bound their rounding)."""
    g, rstd = g.double(), rstd.double()[:, None]
    h = s.double() * rstd
    f = g * w.double()
    dx = rstd * (f - h * (f * h).mean(-1, keepdim=True))
    if gr is not None:
        dx = dx + gr.double()
    return dx, (g * h).sum(0), h, f


def quantize(y):
    """(exact codes before rounding, scale) of rows y."""
    scale = y.double().abs().amax(-1) / 127.0
    return torch.where(scale[:, None] > 0, y.double() / scale[:, None], 0.0), scale


def int8_scores(h, hs, w, ws, b=None):
    """(integer sums as float64, which holds them exactly, and the scores)."""
    s = h.double() @ w.double().T
    z = s * hs.double()[:, None] * ws.double()
    return s, z if b is None else z + b.double()


def cross_entropy(h, w, t, b=None, cap=0.0, row_weight=None, z_loss=0.0):
    """A dict of loss, row, lse, G, dh, dw, db; skipped rows (a target outside [0, V), a weight of 0) count
    nothing and are not read."""
    V = w.shape[0]
    live = (t >= 0) & (t < V)
    if row_weight is not None:
        live &= row_weight != 0
    n = int(live.sum())
    c = torch.where(live, 1.0 / max(n, 1), 0.0).double() if row_weight is None else \
        torch.where(live, row_weight.double(), 0.0)
    x = torch.where(live[:, None], h.double(), 0.0)
    z = x @ w.double().T
    if b is not None:
        z = z + b.double()
    slope = torch.ones_like(z)
    if cap > 0:
        y = torch.tanh(z / cap)
        z, slope = cap * y, 1.0 - y * y
    z = torch.where(torch.isnan(z), -torch.inf, z)
    lse = torch.logsumexp(z, -1)
    at = t.clamp(0, V - 1)[:, None]
    row = lse - z.gather(1, at)[:, 0]
    if z_loss:
        row = row + z_loss * lse * lse
    G = torch.exp(z - lse[:, None]) * (1.0 + 2.0 * z_loss * lse)[:, None]
    G.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=torch.float64))
    G = torch.where(live[:, None], G * slope * c[:, None], 0.0)
    row, lse = torch.where(live, row, 0.0), torch.where(live, lse, 0.0)
    return dict(loss=torch.where(live, c * row, 0.0).sum(), row=row, lse=lse, G=G, dh=G @ w.double(), dw=G.T @ x,
                db=G.sum(0), z=z, live=live, c=c)
