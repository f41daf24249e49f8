"""Refusals of the operators around the block, on the host (no GPU): every invalid call returns its
status before anything is enqueued, and the wrappers refuse tensors that do not fit."""
import ctypes

import pytest
import torch

from tests.conftest import ensure_built

FAKE = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100001)
BIG = 1 << 60
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def nat():
    ensure_built()
    from routing_shared_expert_gb300 import _native
    return _native


def fields(c, kw):
    for k, v in kw.items():
        setattr(c, k, v)
    return c


# ------------------------------------------------------------------------ layer norm --

def norm(nat, **kw):
    return fields(nat.moe_layernorm_config(4, 64, 0, 1e-5, 1, 1, 1, 1, 0, 0, 0, 0), kw)


def forward(nat, c, **kw):
    a = dict(x=FAKE, r=FAKE, w=FAKE, b=FAKE, s=FAKE, y=FAKE, mean=FAKE, rstd=FAKE)
    a.update(kw)
    return nat.library().moe_layernorm_forward(None if c is None else ctypes.byref(c), *a.values(), None)


def backward(nat, c, **kw):
    a = dict(h=FAKE, w=FAKE, mean=FAKE, rstd=FAKE, dy=FAKE, ds=FAKE, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE, n=BIG)
    a.update(kw)
    return nat.library().moe_layernorm_backward(None if c is None else ctypes.byref(c), *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(T=(1 << 30) + 1), -1), (dict(d=0), -1), (dict(d=(1 << 20) + 1), -1), (dict(kind=2), -1),
    (dict(kind=-1), -1), (dict(eps=-1e-6), -1), (dict(eps=NAN), -1), (dict(eps=INF), -1), (dict(x_dtype=2), -1),
    (dict(stream_dtype=-1), -1), (dict(y_dtype=3), -1), (dict(w_dtype=2), -1), (dict(ldx=63), -1), (dict(ldr=1), -1),
    (dict(lds=-64), -1), (dict(ldy=63), -1), (dict(T=1 << 30, d=1 << 20), -2), (dict(ldy=1 << 50), -2),
    (dict(ldx=1 << 62), -2),
])
def test_layernorm_config_refusals(nat, kw, status):
    assert forward(nat, norm(nat, **kw)) == status
    assert backward(nat, norm(nat, **kw)) == status


def test_layernorm_argument_refusals(nat):
    c = norm(nat)
    assert forward(nat, None) == -1 and backward(nat, None) == -1
    for k in ("x", "y"):
        assert forward(nat, c, **{k: None}) == -1
    assert forward(nat, c, r=None) == -1                      # a sum without a residual
    assert forward(nat, norm(nat, kind=1)) == -1              # RMS has no mean
    for k in ("x", "r", "w", "b", "s", "y", "mean", "rstd"):
        assert forward(nat, c, **{k: ODD}) == -7
    for k in ("h", "mean", "rstd", "dy", "ws"):
        assert backward(nat, c, **{k: None}) == -1
    for k in ("h", "w", "mean", "rstd", "dy", "ds", "dx", "dw", "db", "ws"):
        assert backward(nat, c, **{k: ODD}) == -7
    assert backward(nat, c, n=256) == -4
    assert backward(nat, c, ws=ctypes.c_void_p(0x100040)) == -7
    # no rows: nothing to do, nothing enqueued
    none = norm(nat, T=0)
    assert forward(nat, none, x=None, y=None, r=None, s=None) == 0
    assert backward(nat, none, h=None, dy=None, mean=None, rstd=None, dw=None, db=None) == 0
    n = ctypes.c_size_t()
    size = nat.library().moe_layernorm_workspace_size
    assert size(4, 64, None) == -1 and size(-1, 64, ctypes.byref(n)) == -1 and size(4, 0, ctypes.byref(n)) == -1
    assert size(4, (1 << 20) + 1, ctypes.byref(n)) == -1
    assert nat.moe_layernorm_workspace_size(1, 64) < nat.moe_layernorm_workspace_size(4096, 64)


def test_a_single_row_has_no_stride(nat):
    """One row: what the strides say is not looked at, so that no stride of it is refused."""
    c = norm(nat, T=1, ldx=3, ldr=1, lds=5, ldy=-7)
    assert forward(nat, c, y=ODD) == -7 and backward(nat, c, dy=ODD) == -7


# ------------------------------------------------------------------------- embedding --

def emb(nat, **kw):
    return fields(nat.moe_embedding_config(8, 100, 64, 1, 1, 1, 1.0, 0, 0), kw)


def lookup(nat, c, ids=FAKE, table=FAKE, out=FAKE, ws=FAKE, n=BIG):
    return nat.library().moe_embedding_forward(None if c is None else ctypes.byref(c), ids, table, out, ws, n, None)


def gather(nat, c, ids=FAKE, dout=FAKE, dtable=FAKE, acc=0, ws=FAKE, n=BIG):
    return nat.library().moe_embedding_backward(None if c is None else ctypes.byref(c), ids, dout, dtable, acc, ws,
                                                n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(T=(1 << 26) + 1), -1), (dict(V=0), -1), (dict(V=(1 << 30) + 1), -1), (dict(d=0), -1),
    (dict(d=(1 << 20) + 1), -1), (dict(ids_int64=2), -1), (dict(table_dtype=2), -1), (dict(out_dtype=-1), -1),
    (dict(scale=NAN), -1), (dict(scale=-INF), -1), (dict(ldt=63), -1), (dict(ldo=-64), -1),
    (dict(V=1 << 30, d=1 << 20), -2), (dict(ldo=1 << 60), -2), (dict(ldt=1 << 50), -2),
])
def test_embedding_config_refusals(nat, kw, status):
    assert lookup(nat, emb(nat, **kw)) == status
    assert gather(nat, emb(nat, **kw)) == status


def test_embedding_argument_refusals(nat):
    c = emb(nat)
    assert lookup(nat, None) == -1 and gather(nat, None) == -1
    for k in ("ids", "table", "out", "ws"):
        assert lookup(nat, c, **{k: None}) == -1
    for k in ("ids", "dout", "dtable", "ws"):
        assert gather(nat, c, **{k: None}) == -1
    for at in (1, 2, 4):
        assert lookup(nat, c, ids=ctypes.c_void_p(0x100000 + at)) == -7
    for k in ("table", "out", "ws"):
        assert lookup(nat, c, **{k: ODD}) == -7
    for k in ("dout", "dtable", "ws"):
        assert gather(nat, c, **{k: ODD}) == -7
    assert gather(nat, c, acc=2) == -1 and gather(nat, c, acc=-1) == -1
    assert lookup(nat, c, n=255) == -4 and gather(nat, c, n=255) == -4
    none = emb(nat, T=0)
    assert lookup(nat, none, ids=None, out=None, table=None) == 0
    assert gather(nat, none, ids=None, dout=None, dtable=None, acc=1) == 0
    assert gather(nat, none, ids=None, dout=None, dtable=None) == -1     # zeros have to go somewhere
    n = ctypes.c_size_t()
    size = nat.library().moe_embedding_workspace_size
    assert size(8, 100, 64, None) == -1 and size(8, 0, 64, ctypes.byref(n)) == -1
    assert size(8, 100, 64, ctypes.byref(n)) == 0 and n.value % 256 == 0


# ------------------------------------------------------------------------- gradients --

def tensors(nat, *rows):
    return (nat.moe_tensor * max(len(rows), 1))(*[nat.moe_tensor(*r) for r in rows])


def clip(nat, g, out=None, n=None, most=1.0, norm=FAKE, ws=FAKE, b=BIG):
    return nat.library().moe_clip_grad_norm(g, out, len(g) if n is None else n, most, norm, ws, b, None)


A, B = 0x100000, 0x200000


@pytest.mark.parametrize("t,status", [
    ((A, -1, 8, 0, 0), -1), ((A, 1, -8, 0, 0), -1), ((A, 1, 8, 0, 2), -1), ((A, 2, 8, 7, 0), -1),
    ((A, 2, 8, -8, 0), -1), ((None, 1, 8, 0, 0), -1), ((A + 2, 1, 8, 0, 0), -7), ((A + 1, 1, 8, 0, 1), -7),
    ((A, 1 << 30, 1 << 30, 0, 0), -2), ((A, 2, 8, 1 << 41, 0), -2),
])
def test_tensor_refusals(nat, t, status):
    g = tensors(nat, (B, 1, 4, 0, 0), t)
    assert clip(nat, g) == status
    assert nat.library().moe_grad_norm(g, 2, 1.0, FAKE, FAKE, BIG, None) == status


def test_clip_argument_refusals(nat):
    g = tensors(nat, (A, 1, 8, 0, 0))
    assert clip(nat, g, n=-1) == -1 and clip(nat, g, n=(1 << 20) + 1) == -1
    assert clip(nat, g, most=-1.0) == -1 and clip(nat, g, most=NAN) == -1
    assert clip(nat, g, norm=None) == -1 and clip(nat, g, ws=None) == -1
    assert clip(nat, g, norm=ODD) == -7 and clip(nat, g, ws=ctypes.c_void_p(0x100020)) == -7
    assert clip(nat, g, b=256) == -4
    assert nat.library().moe_clip_grad_norm(None, None, 1, 1.0, FAKE, FAKE, BIG, None) == -1
    assert nat.library().moe_grad_norm_workspace_size(None) == -1
    for bad in ((B, 1, 7, 0, 0), (B, 2, 4, 0, 0), (B, 1, 8, 0, 1)):      # another shape or type
        assert clip(nat, g, tensors(nat, bad)) == -1


def test_clip_refuses_outputs_that_share_memory(nat):
    one, two = (A, 1, 8, 0, 0), (B, 1, 8, 0, 0)
    assert clip(nat, tensors(nat, one, one)) == -1                                # twice in place
    assert clip(nat, tensors(nat, one, (A + 28, 1, 8, 0, 0))) == -1
    assert clip(nat, tensors(nat, one, two), tensors(nat, (B + 64, 1, 8, 0, 0), (B + 92, 1, 8, 0, 0))) == -1
    assert clip(nat, tensors(nat, one, two), tensors(nat, two, one)) == -1        # exchanged
    assert clip(nat, tensors(nat, one), tensors(nat, (A + 4, 1, 8, 0, 0))) == -1  # shifted
    # columns of one matrix: apart, and one column too many
    left, right, wide = (A, 4, 8, 16, 0), (A + 32, 4, 8, 16, 0), (A + 28, 4, 8, 16, 0)
    assert clip(nat, tensors(nat, left, wide)) == -1
    assert clip(nat, tensors(nat, right, (A, 4, 9, 16, 0))) == -1
    # what is allowed gets as far as the workspace's own check: nothing is enqueued here
    ok = [(one, (A + 32, 1, 8, 0, 0)), (left, right), (right, left), ((A, 0, 8, 0, 0), (A, 1, 8, 0, 0))]
    for pair in ok:
        assert clip(nat, tensors(nat, *pair), b=256) == -4


# -------------------------------------------------------------------------- wrappers --

class OnDevice(torch.Tensor):
    def get_device(self):
        return 0


class Elsewhere(OnDevice):
    def get_device(self):
        return 1


def dev(t, kind=OnDevice):
    return t.as_subclass(kind)


@pytest.fixture
def here(monkeypatch):
    """Host tensors that say they are on device 0 stand for device tensors; a refused call never looks at
    what their addresses hold."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)


def layernorm_args(**kw):
    a = dict(x=torch.zeros(4, 8), residual=torch.zeros(4, 8), weight=torch.ones(8), bias=torch.ones(8), eps=1e-5,
             sum=torch.zeros(4, 8), y=torch.zeros(4, 8), mean=torch.zeros(4), rstd=torch.zeros(4))
    a.update(kw)
    return {k: dev(v) if type(v) is torch.Tensor else v for k, v in a.items()}


BAD_ROWS = [torch.zeros(4, 7), torch.zeros(8, 4).t(), torch.zeros(4, 8, dtype=torch.float64), torch.zeros(8).expand(4, 8),
            torch.zeros(4, 16)[:, ::2], torch.zeros(4, 8).as_subclass(Elsewhere), torch.zeros(20).as_strided((4, 8), (3, 1))]


@pytest.mark.parametrize("bad", BAD_ROWS)
@pytest.mark.parametrize("which", ["residual", "sum", "y"])
def test_layernorm_refuses_rows_that_do_not_fit(nat, here, which, bad):
    with pytest.raises(ValueError, match=which):
        nat.moe_layernorm_forward(**layernorm_args(**{which: bad}), stream=0)


@pytest.mark.parametrize("kw", [dict(x=torch.zeros(8)), dict(x=torch.zeros(2, 4, 8)), dict(weight=torch.ones(7)),
                                dict(weight=torch.ones(16)[::2]), dict(bias=torch.ones(8, dtype=torch.bfloat16)),
                                dict(weight=torch.ones(8, dtype=torch.float16)), dict(mean=torch.zeros(4, 1)),
                                dict(rstd=torch.zeros(4, dtype=torch.bfloat16)), dict(rstd=torch.zeros(8)),
                                dict(sum=torch.zeros(4, 8, dtype=torch.bfloat16)), dict(kind="batch")])
def test_layernorm_refuses_operands_that_do_not_fit(nat, here, kw):
    with pytest.raises((ValueError, KeyError)):
        nat.moe_layernorm_forward(**layernorm_args(**kw), stream=0)


@pytest.mark.parametrize("which", ["dy", "dsum", "dx"])
@pytest.mark.parametrize("bad", BAD_ROWS)
def test_layernorm_backward_refuses_rows_that_do_not_fit(nat, here, which, bad):
    o = {k: dev(torch.zeros(4, 8)) for k in ("h", "dy", "dsum", "dx")}
    v = {k: dev(torch.zeros(4)) for k in ("mean", "rstd")}
    o[which] = dev(bad) if type(bad) is torch.Tensor else bad
    ws = dev(torch.zeros(1 << 16, dtype=torch.uint8))
    with pytest.raises(ValueError, match=which):
        nat.moe_layernorm_backward(o["h"], None, v["mean"], v["rstd"], o["dy"], o["dsum"], o["dx"], None, None, ws,
                                   stream=0)


def test_embedding_wrapper_refusals(nat, here):
    ids, table, out = dev(torch.zeros(4, dtype=torch.int64)), dev(torch.zeros(10, 8)), dev(torch.zeros(4, 8))
    ws = dev(torch.zeros(256, dtype=torch.uint8))
    for bad in (dict(ids=dev(torch.zeros(4))), dict(ids=dev(torch.zeros(8, dtype=torch.int64)[::2])),
                dict(ids=dev(torch.zeros(5, dtype=torch.int32))), dict(table=dev(torch.zeros(10, 7))),
                dict(table=dev(torch.zeros(8))), dict(out=dev(torch.zeros(8, 4).t())),
                dict(out=dev(torch.zeros(2, 2, 8))), dict(out=dev(torch.zeros(4, 8), Elsewhere)),
                dict(ws=dev(torch.zeros(256, dtype=torch.uint8), Elsewhere)), dict(table=dev(torch.zeros(8).expand(10, 8)))):
        a = dict(ids=ids, table=table, out=out, ws=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            nat.moe_embedding_forward(a["ids"], a["table"], 1.0, a["out"], a["ws"], stream=0)
        with pytest.raises(ValueError):
            nat.moe_embedding_backward(a["ids"], a["out"], 1.0, a["table"], a["ws"], stream=0)


def test_clip_wrapper_refusals(nat, here):
    norm, ws = dev(torch.zeros(2)), dev(torch.zeros(1 << 16, dtype=torch.uint8))
    g = [dev(torch.zeros(4, 8)), dev(torch.zeros(3))]
    for bad in (torch.zeros(4, 8).double(), torch.zeros(8, 4).t(), torch.zeros(8).expand(4, 8), torch.zeros(6)[::2],
                torch.zeros(4, 4, 4).transpose(0, 1)):
        with pytest.raises(ValueError):
            nat.moe_clip_grad_norm([g[0], dev(bad)], 1.0, None, norm, ws, stream=0)
        with pytest.raises(ValueError):
            nat.moe_grad_norm([g[0], dev(bad)], norm, ws, stream=0)
    for out in ([g[0]], [g[1], g[0]], [dev(torch.zeros(8, 4)), g[1]], [g[0], dev(torch.zeros(3).bfloat16())],
                [dev(torch.zeros(8, 4).t()), g[1]]):
        with pytest.raises(ValueError):
            nat.moe_clip_grad_norm(g, 1.0, out, norm, ws, stream=0)
    with pytest.raises(ValueError):
        nat.moe_clip_grad_norm(g, 1.0, None, dev(torch.zeros(1)), ws, stream=0)
    with pytest.raises(nat.MoEError):         # one tensor twice
        nat.moe_clip_grad_norm([g[0], g[0]], 1.0, None, norm, ws, stream=0)


def test_tensors_on_the_host_or_another_device_are_refused(nat, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    x = torch.zeros(4, 8)
    for t in (x, x.as_subclass(Elsewhere)):
        with pytest.raises(ValueError, match="device|CUDA"):
            nat.moe_layernorm_forward(t, None, None, None, 1e-5, None, t, None, None, stream=0)


@pytest.mark.parametrize("d", [1, 64, 2560])
def test_workspaces_hold_calls_of_fewer_tokens(nat, d):
    """A workspace for T tokens is taken for every smaller number of them."""
    tokens = [*range(0, 6000, 7), *range(6000, 60000, 517), *range(131000, 131200), *range(262100, 262200), 1 << 26]
    for V in (1, 1000, 200000):
        sizes = [nat.moe_embedding_workspace_size(T, V, d) for T in tokens]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    sizes = [nat.moe_layernorm_workspace_size(T, d) for T in tokens]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
