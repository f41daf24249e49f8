"""What the wrappers of the block operators refuse before the library sees it (no GPU): operands
whose memory does not hold what the call would read or write.  Host tensors that say they are
on the GPU stand for device tensors; a refused call never looks at what their addresses hold."""
import pytest
import torch

from tests.conftest import ensure_built


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)


def dev(t):
    return t.as_subclass(OnDevice)


@pytest.fixture(scope="module")
def nat():
    ensure_built()
    from routing_shared_expert_gb300 import _native
    return _native


RNG = torch.zeros(2, dtype=torch.int64)


def overlapping(kind, rows, cols):
    """A [rows][cols] matrix whose rows share memory."""
    if kind == "expanded":
        return torch.zeros(cols).expand(rows, cols)
    if kind == "one value":
        return torch.zeros(1, 1).expand(rows, cols)
    return torch.zeros(rows + cols).as_strided((rows, cols), (1, 1))


@pytest.mark.parametrize("kind", ["expanded", "one value", "window"])
@pytest.mark.parametrize("cols", [1, 64])
@pytest.mark.parametrize("which", ["x", "residual", "y", "dy", "dx"])
def test_dropout_refuses_rows_that_overlap(nat, which, cols, kind):
    """A row stride below the row's length: 0 would mean dense rows to the library, which would
    then walk rows * cols elements of a buffer of cols."""
    if kind == "window" and cols == 1:
        return                        # dense: a stride of one element
    rows = 1000
    o = {k: dev(torch.zeros(rows, cols)) for k in ("x", "residual", "y", "dy", "dx")}
    o[which] = dev(overlapping(kind, rows, cols))
    if which in ("x", "residual", "y"):
        with pytest.raises(ValueError, match="rows"):
            nat.moe_dropout_add(o["x"], o["residual"], 0.1, dev(RNG), o["y"], 0)
    else:
        with pytest.raises(ValueError, match="rows"):
            nat.moe_dropout_backward(o["dy"], 0.1, dev(RNG), o["dx"], 0)


def test_dropout_row_strides_that_stay_allowed(nat):
    """Dense, strided and single rows give the library the stride that they have."""
    def shape(t):
        return nat._rows_of("x", dev(t))

    assert shape(torch.zeros(7, 8)) == (7, 8, 8)
    assert shape(torch.zeros(7, 16)[:, :8]) == (7, 8, 16)
    assert shape(torch.zeros(2, 3, 8)) == (6, 8, 8)
    assert shape(torch.zeros(8)) == (1, 8, 8)
    assert shape(torch.zeros(8).expand(1, 8)) == (1, 8, 8)
    assert shape(torch.zeros(7, 3)[:, :1]) == (7, 1, 3)
    assert shape(torch.zeros(0, 8)) == (0, 8, 8)


def layer_cfg(nat):
    return nat.make_config(T=64, d_model=128, N=8, K=2, d_expert=128, d_shared=0, shared_mode="none")


def router_gradient(nat):
    """Every structure of a backward pass through the router, at addresses that nothing looks at."""
    w, o, g = nat.moe_weights(), nat.moe_outputs(), nat.moe_grads()
    for s, names in ((w, ("W_gate", "W_up", "W_down", "W_router")),
                     (o, ("topk_idx", "topk_w", "counts_keep", "offsets", "route_pos", "perm_src", "logits")),
                     (g, ("dx", "dW_gate", "dW_up", "dW_down", "dW_router"))):
        for k in names:
            setattr(s, k, 0x100000)
    return w, o, g


@pytest.mark.parametrize("bad", [torch.zeros(64, 8, dtype=torch.bfloat16), torch.zeros(64, 8, dtype=torch.float64),
                                 torch.zeros(63, 8), torch.zeros(64, 7), torch.zeros(8, 64).t(),
                                 torch.zeros(8).expand(64, 8), torch.zeros(8, 64)])
def test_backward_refuses_logit_gradients_that_do_not_fit(nat, bad):
    w, o, g = router_gradient(nat)
    x, dy, ws = dev(torch.zeros(64, 128, dtype=torch.bfloat16)), dev(torch.zeros(64, 128)), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="dlogits"):
        nat.moe_layer_backward_aux(layer_cfg(nat), w, x, o, dy, dev(bad), g, ws, 0)
    with pytest.raises(ValueError, match="dlogits"):     # on the host
        nat.moe_layer_backward_aux(layer_cfg(nat), w, x, o, dy, torch.zeros(64, 8), g, ws, 0)


def test_backward_refuses_misaligned_logit_gradients(nat):
    import ctypes
    lib, fake, big = nat.library(), ctypes.c_void_p(0x100000), 1 << 60
    w, o, g = router_gradient(nat)
    c = layer_cfg(nat)
    for at in (0x100001, 0x100002, 0x100003):
        assert lib.moe_layer_backward_aux(ctypes.byref(c), ctypes.byref(w), fake, ctypes.byref(o), fake,
                                          ctypes.c_void_p(at), ctypes.byref(g), fake, big, None) == -7
