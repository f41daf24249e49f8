"""The measured cases of the training-block operators around the MoE layer.

Three operators, each with a plain form in elementary torch operations and the call a user
makes of the library:

* ``linear``: y = act(x W^T + b) + r for the projections beside the MoE layer, with its
  backward pass (dx, dW, db from dy and the saved pre-activation);
* ``dropout``: y = r + keep * x / (1 - p) with a keep mask that is never stored: element i
  is kept when word i mod 4 of Philox4x32-10 (Salmon et al., 2011) at counter
  (i div 4, offset) under key ``seed`` is at least round(p 2^32); and its backward pass;
* ``balance``: the router's load-balancing loss over sequences and its z-loss, with the
  per-expert counts and the gradient of the logits.

``own`` chooses the form ``run`` takes: False the plain one, True the library's.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of a decode step through an attention output projection and its residual
        dict(name="linear 1 token", op="linear", T=1, n_in=2048, n_out=2048, act="none", bias=True,
             residual=True, out="bf16", save_pre=False),
        # a small decode batch through the wide projection of a dense feed-forward layer
        dict(name="linear 24 tokens silu", op="linear", T=24, n_in=4096, n_out=14336, act="silu",
             bias=False, residual=False, out="bf16", save_pre=False),
        # a prompt of odd length
        dict(name="linear 1237 tokens gelu", op="linear", T=1237, n_in=2048, n_out=5632,
             act="gelu", bias=True, residual=False, out="bf16", save_pre=False),
        # a training batch through a square projection into an fp32 residual stream
        dict(name="linear 8192 fp32 residual", op="linear", T=8192, n_in=2560, n_out=2560,
             act="none", bias=True, residual=True, out="f32", save_pre=False),
        # the largest training batch: wide projection, pre-activation kept for the backward pass
        dict(name="linear 32768 gelu saved", op="linear", T=32768, n_in=4096, n_out=14336,
             act="gelu_tanh", bias=True, residual=False, out="bf16", save_pre=True),
        # gradients of a short ragged batch into an odd number of features
        dict(name="linear backward odd", op="linear_backward", T=999, n_in=2048, n_out=1407,
             act="silu", bias=True, out="bf16"),
        # gradients of a training batch
        dict(name="linear backward 16384", op="linear_backward", T=16384, n_in=2048, n_out=5632,
             act="gelu_tanh", bias=True, out="bf16"),
        # the smallest layer, fp32 throughout
        dict(name="dropout tiny", op="dropout", rows=256, cols=64, p=0.1, x="f32", res="f32",
             out="f32"),
        # a layer's fp32 output dropped out and added to a bf16 residual stream
        dict(name="dropout add 8192", op="dropout", rows=8192, cols=7168, p=0.1, x="f32",
             res="bf16", out="bf16"),
        # its gradient, on an odd shape, in the fp32 that the layer's backward pass takes
        dict(name="dropout backward odd", op="dropout_backward", rows=16383, cols=2047, p=0.05,
             x="bf16", out="f32"),
        # the smallest router
        dict(name="balance tiny", op="balance", T=256, N=8, K=2, score="softmax", seq_len=0,
             masked=False, z=0.001),
        # 32 sequences through a 256-expert sigmoid router, padding masked
        dict(name="balance 131072 sequences", op="balance", T=131072, N=256, K=8, score="sigmoid",
             seq_len=4096, masked=True, z=0.001),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "dropout", "dropout_backward", "balance"])
    if op.startswith("linear"):
        while True:
            T, n_in, n_out = _log_int(rng, 1, 32768), _log_int(rng, 64, 14336), _log_int(rng, 64, 14336)
            if rng.random() < 0.8:      # most models keep their widths at multiples of 64
                n_in = (n_in + 63) // 64 * 64
            if rng.random() < 0.7:
                n_out = (n_out + 63) // 64 * 64
            if T * n_in * n_out <= 16384 * 4096 * 14336:
                break
        c = dict(op=op, T=T, n_in=n_in, n_out=n_out,
                 act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                 bias=rng.random() < 0.7)
        if op == "linear":
            c.update(residual=rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "f32"]),
                     save_pre=rng.random() < 0.3)
        else:
            c.update(out=rng.choice(["bf16", "bf16", "f32"]))
        return c
    if op.startswith("dropout"):
        while True:
            rows, cols = _log_int(rng, 1, 32768), _log_int(rng, 64, 14336)
            if rng.random() < 0.6:
                cols = (cols + 63) // 64 * 64
            if rows * cols <= 8192 * 7168:
                break
        c = dict(op=op, rows=rows, cols=cols, p=rng.choice([0.0, 0.05, 0.1, 0.25, 0.5]),
                 x=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
        if op == "dropout":
            c["res"] = rng.choice(["none", "bf16", "f32"])
        return c
    T = _log_int(rng, 1, 131072)
    N = rng.choice([8, 32, 60, 64, 128, 160, 256, rng.randint(1, 255)])
    return dict(op="balance", T=T, N=N, K=rng.randint(1, min(N, 8)),
                score=rng.choice(["softmax", "sigmoid"]),
                seq_len=rng.choice([0, _log_int(rng, min(T, 128), T)]),
                masked=rng.random() < 0.5, z=rng.choice([0.0, 0.001]))


# ----------------------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"].startswith("linear"):
        T, n_in, n_out, out = case["T"], case["n_in"], case["n_out"], DTYPES[case["out"]]
        s["x"] = _normal(g, (T, n_in), 1.0, torch.bfloat16)
        s["W"] = _normal(g, (n_out, n_in), 0.02, torch.bfloat16)
        s["bias"] = _normal(g, (n_out,), 0.1, torch.float32) if case["bias"] else None
        if case["op"] == "linear":
            s["residual"] = _normal(g, (T, n_out), 1.0, out) if case["residual"] else None
            s["y"] = torch.empty((T, n_out), dtype=out, device="cuda")
            s["pre"] = torch.empty_like(s["y"]) if case["save_pre"] else None
        else:
            # what the forward pass saved, and the gradient of its output
            z = s["x"] @ s["W"].t()
            s["pre"] = (z if s["bias"] is None else z + s["bias"]).to(out)
            s["dy"] = _normal(g, (T, n_out), 1e-3, out)
            s["dx"] = torch.empty_like(s["x"])
            s["dW"] = torch.empty_like(s["W"])
            s["dbias"] = torch.empty((n_out,), device="cuda")
    elif case["op"].startswith("dropout"):
        shape = (case["rows"], case["cols"])
        s["x"] = _normal(g, shape, 1.0, DTYPES[case["x"]])
        res = case.get("res", "none")
        s["residual"] = _normal(g, shape, 1.0, DTYPES[res]) if res != "none" else None
        s["y"] = torch.empty(shape, dtype=DTYPES[case["out"]], device="cuda")
        # seed and offset of the generator
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device="cuda")
    else:
        T, N, K = case["T"], case["N"], case["K"]
        # tokens around per-expert popularities, as a router in training has them
        popular = 0.5 * torch.randn((1, N), generator=g, device="cuda")
        s["logits"] = torch.randn((T, N), generator=g, device="cuda") + popular
        s["topk"] = torch.topk(s["logits"], K, dim=1).indices.to(torch.int32)
        s["mask"] = None
        if case["masked"]:      # padding at the end of each sequence
            L = case["seq_len"] or T
            keep = 1 + (torch.rand((-(-T // L),), generator=g, device="cuda") * 0.3 + 0.7) * (L - 1)
            pos = torch.arange(T, device="cuda")
            s["mask"] = (pos % L < keep[pos // L]).to(torch.uint8)
        S = -(-T // (case["seq_len"] or T))
        s["counts"] = torch.empty((S, N), dtype=torch.int32, device="cuda")
        s["P"] = torch.empty((S, N), device="cuda")
        s["loss"] = torch.empty((3,), device="cuda")
        s["dlogits"] = torch.empty((T, N), device="cuda")
    return s


COEF_BALANCE = 0.01


# -------------------------------------------------------------------------- plain form --

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    return torch.ones_like(z)


def _plain_linear(s):
    z = s["x"].float() @ s["W"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(s["y"].dtype)}
    if s["pre"] is not None:
        out["pre"] = z.to(s["pre"].dtype)
    return out


def _plain_linear_backward(s):
    dz = s["dy"].float() * _act_grad(s["pre"].float(), s["case"]["act"])
    out = {"dx": (dz @ s["W"].float()).to(s["dx"].dtype),
           "dW": (dz.t() @ s["x"].float()).to(s["dW"].dtype)}
    if s["bias"] is not None:
        out["dbias"] = dz.sum(0)
    return out


def _philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 on words held in int64 (the high word of a product is the product
    shifted, whatever its sign)."""
    low = 0xFFFFFFFF
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _plain_dropout(s):
    x, p, rng = s["x"], s["case"]["p"], s["rng"]
    n = x.numel()
    q = torch.arange((n + 3) // 4, device=x.device)
    low = 0xFFFFFFFF
    seed, offset = rng[0], rng[1]
    words = _philox(q & low, q >> 32, (offset & low).expand_as(q), ((offset >> 32) & low).expand_as(q),
                    seed & low, (seed >> 32) & low)
    keep = torch.stack(words, 1).view(-1)[:n].view(x.shape) >= int(p * 2.0 ** 32 + 0.5)
    y = torch.where(keep, x.float() * (1 / (1 - p)), torch.zeros((), device=x.device))
    if s["residual"] is not None:
        y = s["residual"].float() + y
    return {"y": y.to(s["y"].dtype)}


def _plain_balance(s):
    case, z, idx = s["case"], s["logits"], s["topk"]
    T, N, K = case["T"], case["N"], case["K"]
    L = case["seq_len"] or T
    S = -(-T // L)
    dev = z.device
    seq = torch.arange(T, device=dev) // L
    on = torch.ones((T,), device=dev) if s["mask"] is None else (s["mask"] != 0).float()
    # requests of each expert by the tokens of each sequence
    flat = (seq[:, None] * N + idx.long()).view(-1)
    counts = torch.zeros((S * N,), dtype=torch.int64, device=dev)
    counts = counts.scatter_add_(0, flat, on.to(torch.int64)[:, None].expand(T, K).reshape(-1)).view(S, N)
    per_seq = lambda v: torch.cat([v, v.new_zeros((S * L - T,) + v.shape[1:])]).view((S, L) + v.shape[1:]).sum(1)  # noqa: E731
    valid = per_seq(on)
    total, nonempty = valid.sum().clamp(min=1), (valid > 0).sum().clamp(min=1).float()
    # scores normalised over the experts
    m = z.max(1, keepdim=True).values
    e = torch.exp(z - m)
    soft = e / e.sum(1, keepdim=True)
    lse = (m + torch.log(e.sum(1, keepdim=True)))[:, 0]
    sig = 1 / (1 + torch.exp(-z))
    p = soft if case["score"] == "softmax" else sig / sig.sum(1, keepdim=True)
    nv = valid.clamp(min=1)
    P = per_seq(p * on[:, None]) / nv[:, None]
    # f - 1/N from the whole counts: the scores sum to one, so the constant drops out
    dev_f = (N * counts.double() - K * valid.double()[:, None]) / (N * K * nv.double()[:, None])
    l_bal = ((1 + N * (dev_f * P).sum(1)) * (valid > 0)).sum() / nonempty
    l_z = (lse * lse * on).double().sum() / total
    f = dev_f.float()[seq]
    d = p * (f - (f * p).sum(1, keepdim=True))
    if case["score"] == "sigmoid":
        d = d * (1 - sig)
    dz = (COEF_BALANCE * N / nonempty / nv)[seq][:, None] * d
    dz = dz + (2 * case["z"] / total) * lse[:, None] * soft
    dz = torch.where(on[:, None] > 0, dz, torch.zeros((), device=dev))
    loss = torch.stack([COEF_BALANCE * l_bal + case["z"] * l_z, l_bal.double(), l_z.double()])
    return {"counts": counts.to(torch.int32), "P": P, "loss": loss.float(), "dlogits": dz}


# ------------------------------------------------------------------- the library's form --

def _own(s):
    import routing_shared_expert_gb300 as moe
    case = s["case"]
    if case["op"].startswith("linear"):
        if "cfg" not in s:      # the plan a program keeps: the configuration and its workspace
            s["cfg"] = moe.make_linear_config(T=case["T"], in_features=case["n_in"],
                                              out_features=case["n_out"], act=case["act"],
                                              out_dtype=case["out"])
            s["ws"] = moe.alloc_linear_workspace(s["cfg"])
        if case["op"] == "linear":
            moe.moe_linear_forward(s["cfg"], s["x"], s["W"], s["bias"], s["residual"], s["pre"],
                                   s["y"], s["ws"])
            return {"y": s["y"]} if s["pre"] is None else {"y": s["y"], "pre": s["pre"]}
        db = s["dbias"] if s["bias"] is not None else None
        moe.moe_linear_backward(s["cfg"], s["x"], s["W"], s["pre"], s["dy"], s["dx"], s["dW"], db,
                                s["ws"])
        return {"dx": s["dx"], "dW": s["dW"]} if db is None else {"dx": s["dx"], "dW": s["dW"], "dbias": db}
    if case["op"] == "dropout":
        moe.moe_dropout_add(s["x"], s["residual"], case["p"], s["rng"], s["y"])
        return {"y": s["y"]}
    if case["op"] == "dropout_backward":
        moe.moe_dropout_backward(s["x"], case["p"], s["rng"], s["y"])
        return {"y": s["y"]}
    if "cfg" not in s:
        s["cfg"] = moe.make_config(T=case["T"], d_model=2048, N=case["N"], K=case["K"], d_expert=2048,
                                   d_shared=0, score=case["score"], shared_mode="none")
        s["ws"] = moe.alloc_balance_loss_workspace(s["cfg"], case["seq_len"])
    moe.moe_balance_loss(s["cfg"], s["logits"], s["topk"], s["mask"], case["seq_len"], COEF_BALANCE,
                         case["z"], None, s["counts"], s["P"], s["loss"], s["dlogits"], s["ws"])
    return {k: s[k] for k in ("counts", "P", "loss", "dlogits")}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "linear":
        return _plain_linear(state)
    if op == "linear_backward":
        return _plain_linear_backward(state)
    if op.startswith("dropout"):
        return _plain_dropout(state)
    return _plain_balance(state)


# ------------------------------------------------------------------------------- work --

def work(case):
    if case["op"].startswith("linear"):
        T, n_in, n_out, o = case["T"], case["n_in"], case["n_out"], BYTES[case["out"]]
        operands = 2 * (T * n_in + n_out * n_in)
        if case["op"] == "linear":
            rows = 1 + bool(case["residual"]) + bool(case["save_pre"])
            return {"bytes": operands + 4 * n_out * bool(case["bias"]) + rows * o * T * n_out,
                    "flops": 2.0 * T * n_in * n_out}
        rows = 1 if case["act"] == "none" else 2        # dy, and the saved pre-activation
        return {"bytes": 2 * operands + 4 * n_out * bool(case["bias"]) + rows * o * T * n_out,
                "flops": 4.0 * T * n_in * n_out}
    if case["op"].startswith("dropout"):
        n = case["rows"] * case["cols"]
        res = case.get("res", "none")
        return {"bytes": n * (BYTES[case["x"]] + BYTES[case["out"]] + (BYTES[res] if res != "none" else 0)) + 16,
                "flops": 2.0 * n}
    T, N, K = case["T"], case["N"], case["K"]
    S = -(-T // (case["seq_len"] or T))
    return {"bytes": 8 * T * N + 4 * T * K + T * bool(case["masked"]) + 8 * S * N + 12,
            "flops": 12.0 * T * N}


# ------------------------------------------------------------------------------ exact --

def _philox_numpy(n, seed, offset):
    """The first n words of the counter sequence, in numpy's unsigned integers."""
    u64, low = np.uint64, np.uint64(0xFFFFFFFF)
    q = np.arange((n + 3) // 4, dtype=u64)
    ctr = [q & low, q >> u64(32), np.full_like(q, offset & 0xFFFFFFFF), np.full_like(q, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        lo_hi = []
        for mult, word in ((0xD2511F53, ctr[0]), (0xCD9E8D57, ctr[2])):
            prod = word * u64(mult)
            lo_hi.append((prod & low, prod >> u64(32)))
        (lo0, hi0), (lo1, hi1) = lo_hi
        ctr = [hi1 ^ ctr[1] ^ u64(key[0]), lo1, hi0 ^ ctr[3] ^ u64(key[1]), lo0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    return np.stack([c.astype(np.uint32) for c in ctr], axis=1).reshape(-1)[:n]


def _phi(z):
    """The normal distribution function."""
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("linear"):
        act = case["act"]
        x, W = s["x"].double(), s["W"].double()
        if case["op"] == "linear":
            z = torch.einsum("ti,oi->to", x, W)
            if s["bias"] is not None:
                z += s["bias"].double()
            y = {"none": lambda: z, "relu": lambda: z.clamp(min=0), "gelu": lambda: z * _phi(z),
                 "gelu_tanh": lambda: z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)),
                 "silu": lambda: z * torch.sigmoid(z)}[act]()
            if s["residual"] is not None:
                y = y + s["residual"].double()
            return {"y": y, "pre": z} if s["pre"] is not None else {"y": y}
        z = s["pre"].double()
        if act == "none":
            slope = torch.ones_like(z)
        elif act == "relu":
            slope = (z > 0).double()
        elif act == "gelu":
            slope = _phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        elif act == "gelu_tanh":
            g = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
            slope = g + z * g * (1 - g) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)
        else:
            g = torch.sigmoid(z)
            slope = g + z * g * (1 - g)
        dz = s["dy"].double() * slope
        out = {"dx": torch.einsum("to,oi->ti", dz, W), "dW": torch.einsum("to,ti->oi", dz, x)}
        if s["bias"] is not None:
            out["dbias"] = dz.sum(dim=0)
        return out
    if case["op"].startswith("dropout"):
        x = s["x"].double()
        rng = [int(v) for v in s["rng"].tolist()]
        words = _philox_numpy(x.numel(), rng[0], rng[1])
        keep = torch.from_numpy(words >= round(case["p"] * 2 ** 32)).to(x.device).view(x.shape)
        y = keep.double() * x / (1 - case["p"])
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    # balance: sequence by sequence
    T, N, K = case["T"], case["N"], case["K"]
    L = case["seq_len"] or T
    z, idx = s["logits"].double(), s["topk"].long()
    on = torch.ones((T,), dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"].bool()
    spans = [(a, min(a + L, T)) for a in range(0, T, L)]
    total = max(1, int(on.sum()))
    nonempty = max(1, sum(int(on[a:b].any()) for a, b in spans))
    Ps, l_bal = [], 0.0
    dz = torch.zeros_like(z)
    counts = []
    for a, b in spans:
        o, zz = on[a:b], z[a:b]
        n = int(o.sum())
        c = torch.bincount(idx[a:b][o].reshape(-1), minlength=N).double()
        counts.append(c)
        if n == 0:
            Ps.append(torch.zeros_like(c))
            continue
        if case["score"] == "softmax":
            p, chain = torch.softmax(zz, dim=1), 1.0
        else:
            g = torch.sigmoid(zz)
            p, chain = g / g.sum(dim=1, keepdim=True), 1 - g
        f = c / (K * n)
        P = p[o].mean(dim=0)
        Ps.append(P)
        l_bal += N * float((f * P).sum()) / nonempty
        d = p * chain * (f - (p @ f)[:, None]) * (COEF_BALANCE * N / (nonempty * n))
        dz[a:b] = d * o[:, None]
    lse = torch.logsumexp(z, dim=1)
    l_z = float((lse[on] ** 2).sum()) / total
    dz += torch.softmax(z, dim=1) * (2 * case["z"] / total * lse * on)[:, None]
    loss = torch.tensor([COEF_BALANCE * l_bal + case["z"] * l_z, l_bal, l_z], dtype=torch.float64)
    return {"counts": torch.stack(counts), "P": torch.stack(Ps), "loss": loss, "dlogits": dz}
