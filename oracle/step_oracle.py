"""float64 oracles of the operators around the block: normalisation of rows with its gradients, token
embedding with its gradient, and the global gradient norm with clipping.

Torch float64 on the device of the inputs; elementwise error bounds of the library's kernels stand
beside the values they bound.  u = 2^-24 is half a step of fp32, relative."""
import math

import torch

from oracle.block_oracle import EPS32 as U
from oracle.block_oracle import half_step


def _depth(n):
    """Additions on the way of one of n values into a row's sum: a thread's own of n / 128 at most (the
    narrowest CTA that takes a row of many values), 32 at least, then two rounds of five over lanes and warps."""
    return max(32, n // 128) + 12


def _rounded(v, e, dtype):
    """Bound of the error of v, known within e, after a rounding to dtype; values below the normal range are
    within one smallest normal."""
    return e + half_step(dtype) * (v.abs() + e) + torch.finfo(dtype).tiny


def layernorm(x, residual, weight, bias, eps, kind, sum_dtype, y_dtype):
    """{name: (value, bound of its error)} of sum, mean, rstd and y.  sum_dtype: the type in which the sum is
    stored before it is normalised, None where it is not."""
    h = x.double()
    d = h.shape[1]
    D = _depth(d)
    out = {}
    eh = torch.zeros_like(h)
    if residual is not None:
        total = h + residual.double()
        if sum_dtype is not None:
            # exactly what a sum in fp32, rounded to the stored type, holds
            h = (x.float() + residual.float()).to(sum_dtype).double()
            out["sum"] = (total, _rounded(total, U * total.abs(), sum_dtype))
        else:
            h, eh = total, U * total.abs()
    if kind == "layer":
        mean = h.mean(1, keepdim=True)
        em = (D + 2) * U * h.abs().mean(1, keepdim=True) + eh.mean(1, keepdim=True)
    else:
        mean, em = torch.zeros_like(h[:, :1]), torch.zeros_like(h[:, :1])
    c = h - mean
    ec = em + eh + U * (c.abs() + em + eh)
    var = (c * c).mean(1, keepdim=True)
    # each square by twice its deviation's error; the squares, their sum and the division
    ev = (2 * c.abs() * ec + ec * ec).mean(1, keepdim=True) + (D + 4) * U * (var + (ec * ec).mean(1, keepdim=True))
    rel = (ev + 2.0 ** -149) / (var + eps)
    rstd = (var + eps) ** -0.5
    er = rstd * (0.5 * rel + rel * rel + 6 * U)
    n = c * rstd
    en = ec * rstd + (c.abs() + ec) * er + U * n.abs()
    w = weight.double() if weight is not None else torch.ones(d, dtype=h.dtype, device=h.device)
    y = n * w
    ey = en * w.abs() + 2 * U * (y.abs() + en * w.abs())
    if bias is not None:
        y = y + bias.double()
        ey = ey + U * (y.abs() + ey)
    out["mean"] = (mean[:, 0], em[:, 0] + U * mean[:, 0].abs())
    out["rstd"] = (rstd[:, 0], er[:, 0])
    out["y"] = (y, _rounded(y, ey, y_dtype))
    return out


def layernorm_backward(h, weight, mean, rstd, dy, dsum, kind, dx_dtype):
    """{name: (value, bound of its error)} of dx, dweight and dbias for the saved statistics."""
    h, dy, r = h.double(), dy.double(), rstd.double()[:, None]
    T, d = h.shape
    D = _depth(d)
    xhat = (h - mean.double()[:, None] if kind == "layer" else h) * r
    w = weight.double() if weight is not None else torch.ones(d, dtype=h.dtype, device=h.device)
    g = dy * w
    c1 = g.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(g[:, :1])
    e1 = (D + 3) * U * g.abs().mean(1, keepdim=True)
    c2 = (g * xhat).mean(1, keepdim=True)
    e2 = (D + 6) * U * (g * xhat).abs().mean(1, keepdim=True)
    dx = r * (g - c1 - xhat * c2)
    size = g.abs() + c1.abs() + (xhat * c2).abs() + e1 + xhat.abs() * e2
    e = r * (e1 + xhat.abs() * e2 + 8 * U * size)
    if dsum is not None:
        dx = dx + dsum.double()
        e = e + U * (dx.abs() + e)
    sums = (T + 8) * U
    return {"dx": (dx, _rounded(dx, e, dx_dtype)),
            "dweight": ((dy * xhat).sum(0), sums * (dy * xhat).abs().sum(0) + 2.0 ** -126),
            "dbias": (dy.sum(0), sums * dy.abs().sum(0) + 2.0 ** -126)}


def embedding(ids, table, scale, out_dtype):
    """(out, bound of its error); the scale reaches the kernel in fp32."""
    ids = ids.reshape(-1).long()
    on = (ids >= 0) & (ids < table.shape[0])
    rows = table.double()[ids.clamp(0, table.shape[0] - 1)] * scale
    rows = torch.where(on[:, None], rows, torch.zeros((), dtype=torch.float64, device=rows.device))
    return rows, torch.where(on[:, None], _rounded(rows, 2 * U * rows.abs(), out_dtype), rows)


def embedding_backward(ids, dout, scale, V, dtype, held=None):
    """(dtable, bound of its error); held: what dtable holds where the sums are added to it."""
    ids = ids.reshape(-1).long()
    on = torch.nonzero((ids >= 0) & (ids < V)).squeeze(1)
    d = dout.shape[-1]
    rows = dout.reshape(-1, d)[on].double()
    zero = torch.zeros((V, d), dtype=torch.float64, device=dout.device)
    n = torch.bincount(ids[on], minlength=V)[:, None].double()
    v = zero.index_put((ids[on],), rows, accumulate=True) * scale
    size = zero.index_put((ids[on],), rows.abs(), accumulate=True) * abs(scale)
    e = (n + 4) * U * size
    none = n == 0
    if held is not None:
        v = v + held.double()
        e = e + U * v.abs()
    bound = torch.where(none, torch.zeros_like(e), _rounded(v, e, dtype))     # without a token: exact
    return v, bound


def grad_norm(grads, max_norm):
    """(norm, coefficient, relative bound of the norm's error, of the coefficient's)."""
    squares, n = 0.0, 0
    for g in grads:
        squares += float((g.double() ** 2).sum())
        n += g.numel()
    norm = math.sqrt(squares)
    coef = 1.0 if math.isinf(max_norm) else max_norm / (norm + 1e-6)
    coef = 1.0 if coef > 1.0 else coef
    # a thread adds at most 64 squares to one sum before that joins another, or n over all threads' worth
    rel = (64 + n / (152 * 256) + 16) * U / 2 + 2 * U
    return norm, coef, rel, rel + 4 * U


def clip(grads, max_norm):
    """[(value, bound of its error)] of the scaled gradients."""
    _, coef, _, rel = grad_norm(grads, max_norm)
    out = []
    for g in grads:
        v = g.double() * coef
        out.append((v, _rounded(v, (rel + U) * v.abs(), g.dtype)))
    return out
