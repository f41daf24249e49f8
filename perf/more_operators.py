"""The measured cases of the operators that a training step puts around the block: the
normalisation in front of it, the token embedding under it, and the gradient norm behind it.

* ``layernorm``: y = (h - mean) rstd w + b of rows h = x + r (the residual stream, stored), or of
  x alone; ``rms`` leaves the mean out.  Its backward pass gives the gradient of h, with the
  stream's own gradient added, and those of w and b.
* ``embedding``: out_t = scale * table[id_t], zeros for id -1; its backward pass gives the dense
  gradient of the table.
* ``clip``: the global norm over a list of gradients, and copies scaled by
  min(1, max_norm / (norm + 1e-6)).

``own`` chooses the form ``run`` takes: False the plain one, True the library's.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
MAX_NORM = 1.0


# ------------------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of a decode step: the stream takes a projection's output and is normalised
        dict(name="layernorm 1 token rms", op="layernorm", T=1, d=2048, kind="rms", x="bf16",
             stream="bf16", y="bf16", w="bf16", bias=False, save=False),
        # a prompt of odd length and width, no residual, statistics kept
        dict(name="layernorm 1237 odd", op="layernorm", T=1237, d=4095, kind="layer", x="bf16",
             stream="none", y="bf16", w="f32", bias=True, save=True),
        # a training batch: the MoE layer's fp32 output joins the bf16 stream
        dict(name="layernorm 8192 rms", op="layernorm", T=8192, d=7168, kind="rms", x="f32",
             stream="bf16", y="bf16", w="f32", bias=False, save=True),
        # gradients of a short ragged batch in fp32
        dict(name="layernorm backward odd", op="layernorm_backward", T=999, d=1407, kind="layer",
             x="f32", y="f32", stream="f32", add=True, w="f32", bias=True),
        # gradients of a training batch, the stream's gradient added
        dict(name="layernorm backward 8192 rms", op="layernorm_backward", T=8192, d=2560, kind="rms",
             x="bf16", y="bf16", stream="bf16", add=True, w="f32", bias=False),
        # the largest training batch
        dict(name="layernorm backward 32768", op="layernorm_backward", T=32768, d=4096, kind="layer",
             x="bf16", y="bf16", stream="bf16", add=False, w="f32", bias=True),
        # one decode step of a small batch
        dict(name="embedding 24 tokens", op="embedding", T=24, V=32000, d=4096, table="bf16",
             out="bf16", ids="int64", scaled=False, padded=False),
        # a training batch from fp32 master weights, scaled by sqrt(d), sequences padded
        dict(name="embedding 131072 scaled", op="embedding", T=131072, V=65536, d=2560, table="f32",
             out="bf16", ids="int32", scaled=True, padded=True),
        # a fine-tuning step of a small vocabulary
        dict(name="embedding backward 300", op="embedding_backward", T=300, V=1000, d=256, table="f32",
             out="f32", ids="int64", scaled=False, padded=False),
        # a training batch: natural-language frequencies, fp32 gradient of the table
        dict(name="embedding backward 32768", op="embedding_backward", T=32768, V=65536, d=2560,
             table="f32", out="bf16", ids="int64", scaled=True, padded=True),
        # the gradients of one small block
        dict(name="clip small block", op="clip", blocks=1, d=256, N=16, d_expert=128, d_shared=128,
             V=0, matrices="f32"),
        # the gradients of one large layer as its backward pass writes them
        dict(name="clip large layer", op="clip", blocks=1, d=2560, N=32, d_expert=2560, d_shared=1280,
             V=0, matrices="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi, regular):
    """A width; most models keep theirs at multiples of 64."""
    d = _log_int(rng, lo, hi)
    return min((d + 63) // 64 * 64, hi) if rng.random() < regular else d


def draw(rng):
    op = rng.choice(["layernorm", "layernorm", "layernorm_backward", "layernorm_backward", "embedding",
                     "embedding_backward", "embedding_backward", "clip"])
    if op.startswith("layernorm"):
        while True:
            T, d = _log_int(rng, 1, 65536), _width(rng, 32, 16384, 0.7)
            if T * d <= 32768 * 4096:
                break
        kind = rng.choice(["rms", "layer"])
        c = dict(op=op, T=T, d=d, kind=kind, x=rng.choice(["bf16", "f32"]), y=rng.choice(["bf16", "bf16", "f32"]),
                 w=rng.choice(["bf16", "f32", "none"]), bias=False)
        if c["w"] != "none":
            c["bias"] = kind == "layer" and rng.random() < 0.6
        if op == "layernorm":
            c.update(stream=rng.choice(["none", "bf16", "f32"]), save=rng.random() < 0.6)
        else:
            c.update(stream=rng.choice(["bf16", "f32"]), add=rng.random() < 0.6)
        return c
    if op.startswith("embedding"):
        while True:
            T, V, d = _log_int(rng, 1, 131072), _log_int(rng, 100, 200000), _width(rng, 32, 8192, 0.7)
            if T * d <= 131072 * 2560 and V * d <= 65536 * 2560:
                break
        return dict(op=op, T=T, V=V, d=d, table=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]),
                    ids=rng.choice(["int32", "int64"]), scaled=rng.random() < 0.5, padded=rng.random() < 0.5)
    while True:
        c = dict(op=op, blocks=_log_int(rng, 1, 24), d=_width(rng, 33, 2560, 0.7), N=_log_int(rng, 1, 64),
                 d_expert=_width(rng, 32, 2560, 0.7), d_shared=_width(rng, 32, 2560, 0.7),
                 V=rng.choice([0, _log_int(rng, 100, 65536)]), matrices=rng.choice(["bf16", "f32"]))
        if sum(math.prod(shape) for shape, _ in _grad_shapes(c)) <= 32 * 2560 * 2560 * 3:
            return c


def _grad_shapes(case):
    """(shape, dtype) of every gradient of a stack of blocks: routed and shared experts, router,
    projection with bias, and norm weights; and of an embedding table."""
    d, N, r, s, m = case["d"], case["N"], case["d_expert"], case["d_shared"], case["matrices"]
    block = [((N, r, d), m), ((N, r, d), m), ((N, d, r), m), ((s, d), m), ((s, d), m), ((d, s), m),
             ((N, d), "f32"), ((d, d), m), ((d,), "f32"), ((d,), "f32")]
    return block * case["blocks"] + ([((case["V"], d), m)] if case["V"] else [])


# ----------------------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _stream_rows(g, T, d, dtype):
    """Rows as a residual stream has them: of different sizes, off centre, a few large features."""
    h = torch.randn((T, d), generator=g, device="cuda")
    size = torch.exp(torch.randn((d,), generator=g, device="cuda") * 0.5)
    return (h * size + 0.1 * size).mul_(torch.exp(torch.randn((T, 1), generator=g, device="cuda"))).to(dtype)


def _token_ids(g, case):
    """Token numbers at natural-language frequencies (about 1 / rank), rank by rank anywhere in the
    vocabulary; padding at the end of each sequence of 512."""
    T, V = case["T"], case["V"]
    u = torch.rand((T,), generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(V + 1.0)).long().sub_(1).clamp_(0, V - 1)
    ids = torch.randperm(V, generator=g, device="cuda")[rank]
    if case["padded"]:
        L = min(512, T)
        keep = 1 + (torch.rand((-(-T // L),), generator=g, device="cuda") * 0.5 + 0.5) * (L - 1)
        pos = torch.arange(T, device="cuda")
        ids = torch.where(pos % L < keep[pos // L], ids, torch.full_like(ids, -1))
    return ids.to(getattr(torch, case["ids"]))


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"].startswith("layernorm"):
        T, d, rms = case["T"], case["d"], case["kind"] == "rms"
        s["eps"] = 1e-6 if rms else 1e-5
        wt = DTYPES.get(case["w"])
        s["weight"] = (1 + _normal(g, (d,), 0.1, torch.float32)).to(wt) if wt else None
        s["bias"] = _normal(g, (d,), 0.1, wt) if case["bias"] else None
        if case["op"] == "layernorm":
            s["x"] = _stream_rows(g, T, d, DTYPES[case["x"]])
            stream = DTYPES.get(case["stream"])
            s["residual"] = _stream_rows(g, T, d, stream) if stream else None
            s["sum"] = torch.empty((T, d), dtype=stream, device="cuda") if stream else None
            s["y"] = torch.empty((T, d), dtype=DTYPES[case["y"]], device="cuda")
            s["mean"] = torch.empty((T,), device="cuda") if case["save"] and not rms else None
            s["rstd"] = torch.empty((T,), device="cuda") if case["save"] else None
        else:
            s["h"] = _stream_rows(g, T, d, DTYPES[case["x"]])
            # what the forward pass saved
            h = s["h"].float()
            s["mean"] = None if rms else h.mean(1)
            s["rstd"] = ((h if rms else h - s["mean"][:, None]).square().mean(1) + s["eps"]).rsqrt()
            s["dy"] = _normal(g, (T, d), 1e-3, DTYPES[case["y"]])
            s["dsum"] = _normal(g, (T, d), 1e-3, DTYPES[case["stream"]]) if case["add"] else None
            s["dx"] = torch.empty((T, d), dtype=DTYPES[case["stream"]], device="cuda")
            s["dweight"] = torch.empty((d,), device="cuda") if wt else None
            s["dbias"] = torch.empty((d,), device="cuda") if case["bias"] else None
    elif case["op"].startswith("embedding"):
        T, V, d = case["T"], case["V"], case["d"]
        s["ids"] = _token_ids(g, case)
        s["scale"] = math.sqrt(d) if case["scaled"] else 1.0
        if case["op"] == "embedding":
            s["table"] = _normal(g, (V, d), 0.02, DTYPES[case["table"]])
            s["out"] = torch.empty((T, d), dtype=DTYPES[case["out"]], device="cuda")
        else:
            s["dout"] = _normal(g, (T, d), 1e-3, DTYPES[case["out"]])
            s["dtable"] = torch.empty((V, d), dtype=DTYPES[case["table"]], device="cuda")
    else:
        # gradients of different tensors differ in size
        s["grads"] = [_normal(g, shape, 1e-3 * 3.0 ** (i % 4), DTYPES[t])
                      for i, (shape, t) in enumerate(_grad_shapes(case))]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
        s["norm"] = torch.empty((2,), device="cuda")
    return s


# -------------------------------------------------------------------------- plain form --

def _plain_layernorm(s):
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        out["sum"] = (h + s["residual"].float()).to(s["sum"].dtype)
        h = out["sum"].float()      # the stream as it is stored
    c = h
    if s["case"]["kind"] == "layer":
        mean = h.mean(1)
        c = h - mean[:, None]
        if s["mean"] is not None:
            out["mean"] = mean
    rstd = 1 / torch.sqrt((c * c).mean(1) + s["eps"])
    if s["rstd"] is not None:
        out["rstd"] = rstd
    y = c * rstd[:, None]
    if s["weight"] is not None:
        y = y * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    out["y"] = y.to(s["y"].dtype)
    return out


def _plain_layernorm_backward(s):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = (h if s["mean"] is None else h - s["mean"][:, None]) * rstd
    g = dy if s["weight"] is None else dy * s["weight"].float()
    dx = g - xhat * (g * xhat).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * rstd
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    out = {"dx": dx.to(s["dx"].dtype)}
    if s["dweight"] is not None:
        out["dweight"] = (dy * xhat).sum(0)
    if s["dbias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


def _plain_embedding(s):
    ids = s["ids"].long()
    rows = s["table"][ids.clamp(min=0)].float() * s["scale"]
    rows = torch.where(ids[:, None] >= 0, rows, torch.zeros((), device=rows.device))
    return {"out": rows.to(s["out"].dtype)}


def _plain_embedding_backward(s):
    ids = s["ids"].long()
    rows = torch.where(ids[:, None] >= 0, s["dout"].float(), torch.zeros((), device=ids.device))
    total = torch.zeros(s["dtable"].shape, device=ids.device)
    total = total.index_add_(0, ids.clamp(min=0), rows) * s["scale"]
    return {"dtable": total.to(s["dtable"].dtype)}


def _plain_clip(s):
    # long sums: each tensor's in 32 bits as torch takes it, their sum in 64
    squares = torch.stack([g.float().square().sum() for g in s["grads"]]).double().sum()
    norm = torch.sqrt(squares)
    coef = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0).float()
    out = {"norm": torch.stack([norm.float(), coef])}
    out.update({f"g{i}": (g.float() * coef).to(g.dtype) for i, g in enumerate(s["grads"])})
    return out


# ------------------------------------------------------------------- the library's form --

def _own(s):
    import routing_shared_expert_gb300 as moe
    case, op = s["case"], s["case"]["op"]
    if op == "layernorm":
        moe.moe_layernorm_forward(s["x"], s["residual"], s["weight"], s["bias"], s["eps"], s["sum"], s["y"],
                                  s["mean"], s["rstd"], kind=case["kind"])
        return {k: s[k] for k in ("sum", "mean", "rstd", "y") if s[k] is not None}
    if op == "layernorm_backward":
        if "ws" not in s:       # the workspace that a program keeps
            s["ws"] = moe.alloc_layernorm_workspace(case["T"], case["d"])
        moe.moe_layernorm_backward(s["h"], s["weight"], s["mean"], s["rstd"], s["dy"], s["dsum"], s["dx"],
                                   s["dweight"], s["dbias"], s["ws"], kind=case["kind"])
        return {k: s[k] for k in ("dx", "dweight", "dbias") if s[k] is not None}
    if op.startswith("embedding"):
        if "ws" not in s:
            s["ws"] = moe.alloc_embedding_workspace(case["T"], case["V"], case["d"])
        if op == "embedding":
            moe.moe_embedding_forward(s["ids"], s["table"], s["scale"], s["out"], s["ws"])
            return {"out": s["out"]}
        moe.moe_embedding_backward(s["ids"], s["dout"], s["scale"], s["dtable"], s["ws"])
        return {"dtable": s["dtable"]}
    if "ws" not in s:
        s["ws"] = moe.alloc_grad_norm_workspace()
    moe.moe_clip_grad_norm(s["grads"], MAX_NORM, s["out"], s["norm"], s["ws"])
    return {"norm": s["norm"], **{f"g{i}": t for i, t in enumerate(s["out"])}}


def run(state):
    if own:
        return _own(state)
    return {"layernorm": _plain_layernorm, "layernorm_backward": _plain_layernorm_backward,
            "embedding": _plain_embedding, "embedding_backward": _plain_embedding_backward,
            "clip": _plain_clip}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- work --

def work(case):
    op = case["op"]
    if op == "layernorm":
        T, d, st = case["T"], case["d"], BYTES.get(case["stream"], 0)
        stats = 4 * T * bool(case["save"]) * (1 if case["kind"] == "rms" else 2)
        return {"bytes": T * d * (BYTES[case["x"]] + 2 * st + BYTES[case["y"]]) + stats
                + d * BYTES.get(case["w"], 0) * (1 + bool(case["bias"])),
                "flops": 8.0 * T * d}
    if op == "layernorm_backward":
        T, d, st = case["T"], case["d"], BYTES[case["stream"]]
        rows = BYTES[case["x"]] + BYTES[case["y"]] + st * (1 + bool(case["add"]))
        params = BYTES.get(case["w"], 0) + 4 * (case["w"] != "none") + 4 * bool(case["bias"])
        return {"bytes": T * d * rows + 4 * T * (1 if case["kind"] == "rms" else 2) + d * params,
                "flops": 14.0 * T * d}
    if op.startswith("embedding"):
        T, V, d, ids = case["T"], case["V"], case["d"], 8 if case["ids"] == "int64" else 4
        if op == "embedding":       # each token's row may be the only one of its kind, up to the table
            return {"bytes": T * (d * BYTES[case["out"]] + ids) + _distinct(T, V) * d * BYTES[case["table"]],
                    "flops": 1.0 * T * d}
        return {"bytes": T * (d * BYTES[case["out"]] + ids) + V * d * BYTES[case["table"]], "flops": 1.0 * T * d}
    n = [(math.prod(shape), BYTES[t]) for shape, t in _grad_shapes(case)]
    return {"bytes": sum(2 * k * b for k, b in n) + 8, "flops": 3.0 * sum(k for k, _ in n)}


def _distinct(T, V):
    """Expected number of different tokens among T at frequencies log(1 + 1 / rank) / log(V + 1)."""
    edges = [1, 2, 3, 5, 10, 20, 50, 100, 300, 1000, 3000, 10000, 30000, 100000, 300000]
    edges = [e for e in edges if e <= V] + [V + 1]
    total = 0.0
    for a, b in zip(edges, edges[1:]):      # ranks of about the same frequency together
        share = math.log(b / a) / math.log(V + 1.0) / (b - a)
        total += (b - a) * -math.expm1(T * math.log1p(-min(share, 1 - 1e-12)))
    return int(min(total, T, V))


# ------------------------------------------------------------------------------ exact --

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "layernorm":
        out = {}
        h = s["x"].double()
        if s["residual"] is not None:
            total = h + s["residual"].double()
            out["sum"] = total
            # normalised is the stream as stored: fp32 holds x + r rounded to it, or on the way to bf16
            h = (s["x"].float() + s["residual"].float()).to(s["sum"].dtype).double()
        if case["kind"] == "layer":
            var, mean = torch.var_mean(h, dim=1, correction=0)
            if s["mean"] is not None:
                out["mean"] = mean
            n = (h - mean.unsqueeze(1)) / torch.sqrt(var + s["eps"]).unsqueeze(1)
        else:
            var = torch.einsum("td,td->t", h, h) / case["d"]
            n = h / torch.sqrt(var + s["eps"]).unsqueeze(1)
        if s["rstd"] is not None:
            out["rstd"] = torch.pow(var + s["eps"], -0.5)
        w = s["weight"].double() if s["weight"] is not None else torch.ones(case["d"], dtype=f64, device="cuda")
        b = s["bias"].double() if s["bias"] is not None else torch.zeros(case["d"], dtype=f64, device="cuda")
        out["y"] = torch.addcmul(b, n, w)
        return out
    if case["op"] == "layernorm_backward":
        # the Jacobian of the normalisation on dy w, with the saved statistics
        h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double()
        if s["mean"] is not None:
            h = h - s["mean"].double().unsqueeze(1)
        h *= r.unsqueeze(1)
        out = {}
        if s["dweight"] is not None:
            out["dweight"] = torch.einsum("td,td->d", dy, h)
        if s["dbias"] is not None:
            out["dbias"] = dy.sum(dim=0)
        if s["weight"] is not None:
            dy *= s["weight"].double()
        along = torch.einsum("td,td->t", dy, h) / case["d"]
        dy -= h * along.unsqueeze(1) + (dy.mean(dim=1, keepdim=True) if case["kind"] == "layer" else 0.0)
        dx = dy * r.unsqueeze(1)
        out["dx"] = dx if s["dsum"] is None else dx + s["dsum"].double()
        return {k: out[k] for k in ("dx", "dweight", "dbias") if k in out}
    if case["op"] == "embedding":
        ids = s["ids"].long()
        out = torch.zeros((case["T"], case["d"]), dtype=f64, device="cuda")
        on = torch.nonzero(ids != -1).squeeze(1)
        out[on] = torch.index_select(s["table"], 0, ids[on]).double() * s["scale"]
        return {"out": out}
    if case["op"] == "embedding_backward":
        ids = s["ids"].long()
        on = torch.nonzero(ids != -1).squeeze(1)
        out = torch.zeros((case["V"], case["d"]), dtype=f64, device="cuda")
        out.index_put_((ids[on],), s["dout"][on].double() * s["scale"], accumulate=True)
        return {"dtable": out}
    n2 = 0.0
    for g in s["grads"]:
        flat = g.reshape(-1)
        for a in range(0, flat.numel(), 1 << 27):
            part = flat[a:a + (1 << 27)].double()
            n2 += float(torch.dot(part, part))
    norm = math.sqrt(n2)
    coef = min(1.0, MAX_NORM / (norm + 1e-6))
    out = {"norm": torch.tensor([norm, coef], dtype=f64, device="cuda")}
    out.update({f"g{i}": g.double() * coef for i, g in enumerate(s["grads"])})
    return out
