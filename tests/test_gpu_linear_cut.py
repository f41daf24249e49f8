"""Projections and gradients deep enough that tiles are cut along the depth: partial sums in scratch
memory, arrival counts, the ordered join.  Each case shows that it cut by what it left in the
scratch memory, which only cut tiles touch: the last 76 slots of 256 x 256 floats of the workspace."""
import pytest
import torch

from tests import test_gpu_linear as L
from tests.conftest import ensure_built

pytestmark = pytest.mark.gpu
SLOT = 256 * 256 * 4
SLOTS = 76


class Recorded:
    """The package with workspaces that start full of NaN patterns, and how many scratch slots a call
    has written since."""

    def __init__(self, moe):
        self._moe, self.ws = moe, None

    def __getattr__(self, name):
        return getattr(self._moe, name)

    def alloc_linear_workspace(self, cfg):
        if self.ws is None or self.ws.numel() < self._moe.moe_linear_workspace_size(cfg):
            self.ws = self._moe.alloc_linear_workspace(cfg)
        self.ws[256:].fill_(0xFF)
        return self.ws

    def slots(self):
        tail = self.ws[self.ws.numel() - SLOTS * SLOT:].view(torch.int32).view(SLOTS, -1)
        touched = (tail != -1).any(1)
        # a slot holds every lane's sums of its part, of 256 columns or of 128
        assert ((tail[touched] != -1).sum(1) % (SLOT // 8) == 0).all(), "a partial tile is incomplete"
        return int(touched.sum())


@pytest.fixture()
def moe():
    ensure_built()
    import routing_shared_expert_gb300 as moe
    return Recorded(moe)


def equal(a, b):
    for u, v in zip(a, b):
        assert torch.equal(u, v), "another call in the same workspace differs"


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,n_in,n_out,kw", [
    (2500, 8192, 2056, dict(act="silu")),                         # a round of whole tiles beside 14 cut ones
    (2500, 8192, 2056, dict(residual=False, pre=False, bias=False)),
    (2500, 8192, 2056, dict(act="gelu", in_place=True)),
    (2500, 8192, 2055, dict(act="gelu_tanh")),                    # unaligned rows
    (2500, 8205, 2056, dict(act="relu", pre=False)),              # an odd depth
    (2500, 8192, 2056, dict(ldr=2060, ldy=2072, off=8)),
    (2304, 14336, 1024, dict(act="silu")),                        # no whole round
])
def test_forward(moe, T, n_in, n_out, kw, out):
    first = L.forward(moe, T, n_in, n_out, out=out, **kw)
    assert moe.slots() >= 2, "nothing was cut"
    again = L.forward(moe, T, n_in, n_out, out=out, ws=moe.ws, **kw)
    equal(*[[t for t in r if t is not None] for r in (first, again)])


@pytest.mark.parametrize("dw", ["bf16", "f32"])
@pytest.mark.parametrize("T,n_in,n_out,kw", [
    (6000, 520, 264, dict()),                       # narrow tiles, three parts
    (6000, 2312, 2056, dict()),                     # whole tiles beside cut ones
    (5003, 264, 520, dict(act="none")),             # dy itself
    (9001, 131, 257, dict(act="gelu")),             # unaligned rows, four parts
    (36001, 72, 130, dict()),                       # eight parts
    (8192, 64, 64, dict(out="f32", act="gelu_tanh")),
    (6000, 520, 264, dict(ldx=523, ldy=267, off=1)),
])
def test_weight_gradients(moe, T, n_in, n_out, kw, dw):
    args = dict(dw_dtype=dw, want=("dW", "dbias"), **kw)
    first = L.backward(moe, T, n_in, n_out, **args)
    assert moe.slots() >= 2, "nothing was cut"
    again = L.backward(moe, T, n_in, n_out, **args)
    equal(*[[r[k] for k in args["want"]] for r in (first, again)])


@pytest.mark.parametrize("dx", ["bf16", "f32"])
@pytest.mark.parametrize("T,n_in,n_out,kw", [
    (300, 264, 8192, dict()),
    (2500, 2056, 6000, dict(act="none")),           # whole tiles beside cut ones
    (301, 263, 8195, dict(act="gelu")),
])
def test_input_gradients(moe, T, n_in, n_out, kw, dx):
    args = dict(dx_dtype=dx, want=("dx", "dbias"), **kw)
    first = L.backward(moe, T, n_in, n_out, **args)
    assert moe.slots() >= 2, "nothing was cut"
    again = L.backward(moe, T, n_in, n_out, **args)
    equal(*[[r[k] for k in args["want"]] for r in (first, again)])


def test_cut_products_in_turn_in_one_workspace(moe):
    """Forward and gradients that cut differently, through one workspace without anything between
    them: the counts of one are zero again for the next, and the bits repeat."""
    shapes = [(2500, 8192, 2056, "bf16"), (2304, 14336, 1024, "f32"), (2500, 8192, 520, "bf16")]
    g = torch.Generator(device="cuda").manual_seed(5)
    m = moe._moe
    cases = []
    for T, i, o, out in shapes:
        cfg = m.make_linear_config(T, i, o, out_dtype=out, dw_dtype="f32")
        t = dict(x=L.rows(g, T, i, torch.bfloat16), W=L.rows(g, o, i, torch.bfloat16, std=i ** -0.5),
                 dy=L.rows(g, T, o, L.DT[out]), y=torch.zeros((T, o), dtype=L.DT[out], device="cuda"),
                 dx=torch.zeros((T, i), dtype=torch.bfloat16, device="cuda"), dW=torch.zeros((o, i), device="cuda"),
                 db=torch.zeros(o, device="cuda"))
        cases.append((cfg, t))
    ws = torch.zeros(max(m.moe_linear_workspace_size(c) for c, _ in cases), dtype=torch.uint8, device="cuda")
    names = ("y", "dx", "dW", "db")
    want = None
    for _ in range(4):
        for c, t in cases:
            for k in names:
                t[k].fill_(7.0)
        for c, t in cases:
            m.moe_linear_forward(c, t["x"], t["W"], None, None, None, t["y"], ws)
            m.moe_linear_backward(c, t["x"], t["W"], None, t["dy"], t["dx"], t["dW"], t["db"], ws)
        got = [t[k].clone() for _, t in cases for k in names]
        if want is not None:
            equal(want, got)
        want = got
    assert m.moe_read_status(ws) == 0
    for c, t in cases:
        ref, _, bound, _ = L.B.linear(t["x"], t["W"], None, None, "none", t["y"].dtype)
        L.within("y", t["y"], ref, bound)
        grads = L.B.linear_backward(t["x"], t["W"], None, t["dy"], "none", t["y"].dtype, torch.bfloat16, torch.float32)
        for k, n in (("dx", "dx"), ("dW", "dW"), ("db", "dbias")):
            L.within(n, t[k], *grads[n])
