"""Refusals of the block operators, on the host (no GPU): every invalid call returns its status
before anything is enqueued, and the Python wrappers refuse tensors that do not fit."""
import ctypes

import pytest
import torch

from tests.conftest import ensure_built

FAKE = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100001)
BIG = 1 << 60


@pytest.fixture(scope="module")
def nat():
    ensure_built()
    from routing_shared_expert_gb300 import _native
    return _native


def lin(nat, **kw):
    c = nat.make_linear_config(T=16, in_features=64, out_features=32)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(T=(1 << 28) + 1), -1), (dict(in_features=0), -1), (dict(out_features=0), -1),
    (dict(in_features=(1 << 20) + 1), -1), (dict(dtype=5), -1), (dict(out_dtype=-1), -1),
    (dict(dx_dtype=9), -1), (dict(dw_dtype=2), -1), (dict(act=5), -1), (dict(act=-1), -1),
    (dict(ldx=63), -1), (dict(ldw=1), -1), (dict(ldr=31), -1), (dict(ldy=-64), -1),
    (dict(ldy=1 << 62), -1), (dict(dtype=0), -2), (dict(T=1 << 28, in_features=1 << 20), -2),
])
def test_linear_config_refusals(nat, kw, status):
    n = ctypes.c_size_t(0)
    c = lin(nat, **kw)
    lib = nat.library()
    assert lib.moe_linear_workspace_size(ctypes.byref(c), ctypes.byref(n)) == status
    assert lib.moe_linear_forward(ctypes.byref(c), FAKE, FAKE, None, None, None, FAKE, FAKE, BIG,
                                  None) == status
    assert lib.moe_linear_backward(ctypes.byref(c), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                   BIG, None) == status


def test_linear_argument_refusals(nat):
    lib, c = nat.library(), lin(nat, act=4)
    p = ctypes.byref(c)
    assert lib.moe_linear_workspace_size(p, None) == -1
    assert lib.moe_linear_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == -1

    def fwd(x=FAKE, W=FAKE, bias=None, res=None, pre=None, y=FAKE, ws=FAKE, n=BIG):
        return lib.moe_linear_forward(p, x, W, bias, res, pre, y, ws, n, None)

    def bwd(x=FAKE, W=FAKE, pre=FAKE, dy=FAKE, dx=FAKE, dW=FAKE, db=FAKE, ws=FAKE, n=BIG):
        return lib.moe_linear_backward(p, x, W, pre, dy, dx, dW, db, ws, n, None)

    for k in ("x", "W", "y", "ws"):
        assert fwd(**{k: None}) == -1
    assert fwd(ws=ctypes.c_void_p(0x100010)) == -7
    assert fwd(n=16) == -4
    for k in ("x", "W", "bias", "res", "pre", "y"):
        assert fwd(**{k: ODD}) == -7
    for k in ("pre", "dy", "x", "W", "ws"):
        assert bwd(**{k: None}) == -1
    for k in ("x", "W", "pre", "dy", "dx", "dW", "db"):
        assert bwd(**{k: ODD}) == -7
    assert bwd(n=16) == -4
    # no tokens: nothing to do, and nothing enqueued
    c.T = 0
    assert fwd(x=None, W=None, y=None) == 0
    assert bwd(x=None, W=None, pre=None, dy=None, dW=None, db=None) == 0


def test_linear_workspace_grows_with_the_tokens(nat):
    a, b = (nat.moe_linear_workspace_size(lin(nat, T=t)) for t in (64, 4096))
    assert 256 <= a < b


def drop(nat, **kw):
    c = nat.moe_dropout_config()
    c.rows, c.cols, c.p = 4, 8, 0.1
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), -1), (dict(cols=-1), -1), (dict(p=-0.1), -1), (dict(p=1.5), -1),
    (dict(p=float("nan")), -1), (dict(x_dtype=2), -1), (dict(y_dtype=-1), -1),
    (dict(residual_dtype=7), -1), (dict(ldx=7), -1), (dict(ldy=7), -1), (dict(ldr=7), -1),
    (dict(ldx=-8), -1), (dict(rows=1 << 39), -2), (dict(ldy=1 << 50), -2), (dict(rows=1 << 62, cols=1 << 62), -2),
])
def test_dropout_config_refusals(nat, kw, status):
    lib, c = nat.library(), drop(nat, **kw)
    assert lib.moe_dropout_add(ctypes.byref(c), FAKE, FAKE, FAKE, FAKE, None) == status
    assert lib.moe_dropout_backward(ctypes.byref(c), FAKE, FAKE, FAKE, None) == status


def test_dropout_argument_refusals(nat):
    lib, c = nat.library(), drop(nat)
    p = ctypes.byref(c)
    assert lib.moe_dropout_add(None, FAKE, None, FAKE, FAKE, None) == -1
    assert lib.moe_dropout_add(p, None, None, FAKE, FAKE, None) == -1
    assert lib.moe_dropout_add(p, FAKE, None, None, FAKE, None) == -1
    assert lib.moe_dropout_add(p, FAKE, None, FAKE, None, None) == -1
    for i in range(4):
        args = [FAKE] * 4
        args[i] = ODD
        assert lib.moe_dropout_add(p, *args, None) == -7
    assert lib.moe_dropout_backward(None, FAKE, FAKE, FAKE, None) == -1
    assert lib.moe_dropout_backward(p, FAKE, ctypes.c_void_p(0x100004), FAKE, None) == -7
    for kw in (dict(rows=0), dict(cols=0)):
        assert lib.moe_dropout_add(ctypes.byref(drop(nat, **kw)), None, None, None, None, None) == 0


def layer_cfg(nat, **kw):
    a = dict(T=64, d_model=64, N=8, K=2, d_expert=64, d_shared=0, shared_mode="none")
    a.update(kw)
    return nat.make_config(**a)


def test_balance_loss_refusals(nat):
    lib, c = nat.library(), layer_cfg(nat)
    n = ctypes.c_size_t(0)

    def size(cfg, seq=0):
        return lib.moe_balance_loss_workspace_size(ctypes.byref(cfg), seq, ctypes.byref(n))

    def call(cfg=c, logits=FAKE, idx=FAKE, mask=None, seq=0, cb=0.1, cz=0.0, gs=None, counts=FAKE,
             P=FAKE, loss=FAKE, dz=FAKE, ws=FAKE, b=BIG):
        return lib.moe_balance_loss(ctypes.byref(cfg), logits, idx, mask, seq, cb, cz, gs, counts, P,
                                    loss, dz, ws, b, None)

    assert size(c) == 0 and n.value % 256 == 0
    assert size(c, -1) == -1 and call(seq=-1) == -1
    bad = layer_cfg(nat)
    bad.K = 9
    assert size(bad) == -1 and call(cfg=bad) == -1
    wide = layer_cfg(nat, T=1 << 20)      # 2^20 sequences of one token, 8 experts: too many
    assert size(wide, 1) == -2 and call(cfg=wide, seq=1) == -2
    assert lib.moe_balance_loss_workspace_size(ctypes.byref(c), 0, None) == -1
    assert call(cb=float("nan")) == -1 and call(cz=float("inf")) == -1
    for k in ("logits", "idx", "ws"):
        assert call(**{k: None}) == -1
    for k in ("logits", "idx", "gs", "counts", "P", "loss", "dz"):
        assert call(**{k: ODD}) == -7
    assert call(ws=ctypes.c_void_p(0x100040)) == -7
    assert call(b=256) == -4


def test_aux_gradient_needs_the_router_gradient(nat):
    lib = nat.library()
    c = layer_cfg(nat, d_model=128, d_expert=128)
    w, o, g = nat.moe_weights(), nat.moe_outputs(), nat.moe_grads()
    for s, names in ((w, ("W_gate", "W_up", "W_down")),
                     (o, ("topk_idx", "topk_w", "counts_keep", "offsets", "route_pos", "perm_src")),
                     (g, ("dx", "dW_gate", "dW_up", "dW_down"))):
        for k in names:
            setattr(s, k, 0x100000)
    assert lib.moe_layer_backward_aux(ctypes.byref(c), ctypes.byref(w), FAKE, ctypes.byref(o), FAKE,
                                      FAKE, ctypes.byref(g), FAKE, BIG, None) == -1


def test_wrappers_refuse_tensors_that_do_not_fit(nat):
    c = nat.make_linear_config(T=2, in_features=64, out_features=8)
    x, W, y = (torch.zeros(s, dtype=torch.bfloat16) for s in ((2, 64), (8, 64), (2, 8)))
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        nat.moe_linear_forward(c, x, W, None, None, None, y, ws)
    with pytest.raises(ValueError, match="CUDA"):
        nat.moe_dropout_add(x, None, 0.1, torch.zeros(2, dtype=torch.int64), x)
    with pytest.raises(ValueError, match="CUDA"):
        nat.moe_balance_loss(layer_cfg(nat), torch.zeros(64, 8), None, None, 0, 0.1, 0.0, None, None,
                             None, None, None, ws)
