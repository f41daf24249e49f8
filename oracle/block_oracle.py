"""float64 oracles of the operators around the layer: the dense projection and its gradients,
dropout from the counter-based generator, and the router's balance loss with its gradient.

Torch float64 on the device of the inputs (numpy for the generator's words); elementwise error
bounds of the library's kernels stand beside the values they bound."""
import math

import numpy as np
import torch

EPS32 = 2.0 ** -24                              # half a step of fp32, relative


def half_step(dtype):
    """Largest relative rounding error of a torch dtype."""
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------------- projection --

def act(z, kind):
    if kind == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z)      # NaN stays
    if kind == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if kind == "gelu_tanh":
        return z * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, kind):
    if kind == "relu":
        return 1 - (z <= 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if kind == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


# Largest slope of the activations (the two forms of GELU reach 1.13, SiLU 1.10), and the
# evaluation error of a value or slope per unit of 1 + |z|: the fast exponential is within
# (2 + 1.2 |argument|) 2^-23 of e^argument, where s (1 - s) |argument| <= 0.23 for a sigmoid of
# it (0.5 with the |z| factor of the slope), and a handful of further roundings.
MAX_SLOPE = 1.13
EVAL = 16 * 2.0 ** -23


def _sum_error(n):
    """Relative error bound of an n-term fp32 sum of products: one step per addition (the
    tensor core may truncate), and the roundings beside it."""
    return (n + 8) * 2.0 ** -23


def linear(x, W, bias, residual, kind, out_dtype):
    """(y, pre, bound of y's error, bound of pre's error)."""
    x, W = x.double(), W.double()
    z, size = x @ W.t(), x.abs() @ W.abs().t()
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    dz = _sum_error(x.shape[1]) * size
    y = act(z, kind)
    dy = (MAX_SLOPE * dz + EVAL * (1 + z.abs())) if kind != "none" else dz
    if residual is not None:
        y, dy = y + residual.double(), dy + EPS32 * (y.abs() + residual.double().abs())
    h = half_step(out_dtype)
    return y, z, dy + h * (y.abs() + dy), dz + h * (z.abs() + dz)


def linear_backward(x, W, pre, dy, kind, out_dtype, dx_dtype, dw_dtype):
    """{name: (value, bound of its error)} for dx, dW and dbias."""
    x, W, dy = x.double(), W.double(), dy.double()
    z = pre.double() if pre is not None else torch.zeros_like(dy)
    dz = dy * act_slope(z, kind)
    ez = EVAL * (1 + z.abs()) * dy.abs() if kind != "none" else torch.zeros_like(dz)
    # dz is rounded to bf16 unless it is dy as given
    rz = ez if kind == "none" and out_dtype == torch.bfloat16 else ez + half_step(torch.bfloat16) * (dz.abs() + ez)
    dz_abs = dz.abs() + rz
    T, n = dz.shape
    out = {}
    for name, a, da, b, terms, dt in (
            ("dx", dz, rz, W, n, dx_dtype), ("dW", dz.t(), rz.t(), x, T, dw_dtype)):
        v = a @ b
        e = da @ b.abs() + _sum_error(terms) * ((a.abs() + da) @ b.abs())
        out[name] = (v, e + half_step(dt) * (v.abs() + e))
    out["dbias"] = (dz.sum(0), ez.sum(0) + (T + 8) * EPS32 * dz_abs.sum(0))
    return out


# ---------------------------------------------------------------------------- dropout --

def philox(counters, seed, offset):
    """Philox4x32-10 words [len(counters)][4] (uint32) at the 64-bit counters."""
    u64, low = np.uint64, np.uint64(0xFFFFFFFF)
    q = np.asarray(counters, dtype=u64)
    c = [q & low, q >> u64(32), np.full_like(q, offset & 0xFFFFFFFF), np.full_like(q, (offset >> 32) & 0xFFFFFFFF)]
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        a, b = c[0] * u64(0xD2511F53), c[2] * u64(0xCD9E8D57)
        c = [(b >> u64(32)) ^ c[1] ^ u64(k0), b & low, (a >> u64(32)) ^ c[3] ^ u64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack([w.astype(np.uint32) for w in c], axis=1)


def keep_mask(rows, cols, p, seed, offset):
    """Boolean [rows][cols] keep mask."""
    n = rows * cols
    words = philox(np.arange((n + 3) // 4), seed, offset).reshape(-1)[:n].astype(np.uint64)
    return torch.from_numpy(words >= np.uint64(math.floor(p * 2.0 ** 32 + 0.5))).view(rows, cols)


def dropout(x, residual, p, seed, offset, out_dtype):
    """(y, bound of its error): the scale, the product and the sum are each rounded to fp32."""
    keep = keep_mask(x.shape[0], x.shape[1], p, seed, offset).to(x.device)
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    d = torch.where(keep, x.double() / (1 - p) if p < 1 else zero, zero)
    y = d if residual is None else d + residual.double()
    e = 2 * EPS32 * d.abs() + (EPS32 * (y.abs() + d.abs()) if residual is not None else 0)
    return y, e + half_step(out_dtype) * (y.abs() + e)


# ----------------------------------------------------------------------- balance loss --

def balance_loss(logits, topk_idx, mask, seq_len, score, coef_b, coef_z, N, K, grad_scale=1.0):
    """dict of counts, P, loss (float64) and dlogits with the bounds P_err, loss_err and
    dlogits_err, sequence by sequence from the definition."""
    z = logits.double()
    T = z.shape[0]
    dev = z.device
    L = seq_len if 0 < seq_len < T else max(T, 1)
    on = torch.ones(T, dtype=torch.bool, device=dev) if mask is None else mask.bool()
    on_idx = topk_idx.long()
    spans = [(a, min(a + L, T)) for a in range(0, T, L)]
    V = int(on.sum())
    ne = sum(int(on[a:b].any()) for a, b in spans)
    z = torch.where(on[:, None], z, torch.zeros((), dtype=torch.float64, device=dev))
    some = on & (z > -math.inf).any(1)
    soft, p, chain = torch.zeros_like(z), torch.zeros_like(z), torch.ones_like(z)
    lse = torch.zeros(T, dtype=torch.float64, device=dev)
    soft[some] = torch.softmax(z[some], 1)
    lse[some] = torch.logsumexp(z[some], 1)
    if score == "softmax":
        p = soft
    else:
        # log sigma = -softplus(-z) keeps the ratios where sigma underflows
        ls = torch.nn.functional.logsigmoid(z)
        p[some] = torch.softmax(ls[some], 1)
        chain = torch.sigmoid(-z)
    counts = torch.zeros((len(spans), N), dtype=torch.int64, device=dev)
    P = torch.zeros((len(spans), N), dtype=torch.float64, device=dev)
    dz, size = torch.zeros_like(z), torch.zeros_like(z)
    l_b = 0.0
    for s, (a, b) in enumerate(spans):
        o = on[a:b]
        v = int(o.sum())
        idx = on_idx[a:b][o].reshape(-1)
        idx = idx[(idx >= 0) & (idx < N)]
        counts[s] = torch.bincount(idx, minlength=N)
        if v == 0:
            continue
        f = counts[s].double() / (K * v)
        pp = p[a:b]
        P[s] = pp[o].mean(0)
        l_b += N * float((f * P[s]).sum()) / ne
        k = grad_scale * coef_b * N / (ne * v)
        # f - f.p for a p that sums to one, against f - 1/N in whole numbers
        d = (N * counts[s] - K * v).double() / (N * K * v)
        dz[a:b] = k * pp * chain[a:b] * (d - (pp @ d)[:, None]) * o[:, None]
        size[a:b] = abs(k) * pp * (d.abs() + (pp @ d.abs())[:, None]) * o[:, None]
    kz = 2 * grad_scale * coef_z / max(V, 1)
    dz += kz * lse[:, None] * soft * on[:, None]
    l_z = float((lse ** 2).sum()) / max(V, 1)
    finite = torch.where(torch.isfinite(z), z, torch.zeros((), dtype=torch.float64, device=dev))
    reach = finite.abs().max(1).values if N else lse
    # relative error of a score: the exponent's argument, its exponential, N additions, a quotient
    rel = (N + 64 + 4 * reach) * EPS32
    size += abs(kz) * (reach + math.log(max(N, 2)))[:, None] * soft * on[:, None]
    worst = float(rel.max()) if T else 0.0
    n_terms = max((b - a for a, b in spans), default=0)
    loss = torch.tensor([coef_b * l_b + coef_z * l_z, l_b, l_z], dtype=torch.float64)
    scale_z = float(((reach + math.log(max(N, 2))) ** 2 * on).sum()) / max(V, 1) if T else 0.0
    e_b, e_z = (worst + (n_terms + N) * EPS32) * abs(l_b), (2 * worst + T * EPS32) * scale_z
    loss_err = torch.tensor([abs(coef_b) * e_b + abs(coef_z) * e_z, e_b, e_z], dtype=torch.float64) \
        + 2 * EPS32 * loss.abs()
    return {"counts": counts, "P": P, "loss": loss, "dlogits": dz,
            "P_err": (worst + (n_terms + 8) * EPS32) * P, "loss_err": loss_err,
            # subnormal results may be flushed or lose bits: one smallest normal
            "dlogits_err": rel[:, None] * size + 2.0 ** -126}
