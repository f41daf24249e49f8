"""A token whose values are broken shows: a NaN reaches every result that depends on it, whatever its
neighbours hold, and nothing else."""
import pytest
import torch

from tests import test_gpu_balance_loss as BL
from tests.conftest import ensure_built

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def moe():
    ensure_built()
    import routing_shared_expert_gb300 as moe
    return moe


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N", [5, 8, 32, 100, 128, 256])
@pytest.mark.parametrize("kind", ["all", "one", "beside -inf", "beside large", "all beside a large row"])
@pytest.mark.parametrize("seq", [64, 0])
def test_balance_loss(moe, score, N, kind, seq):
    T, bad = 6000 if seq == 0 else 320, 69
    z, idx = BL.batch(T, N, 2)
    row = z[bad]
    if kind.startswith("all"):
        row[:] = NAN
    elif kind == "one":
        row[N - 1] = NAN
    elif kind == "beside -inf":
        row[:] = -INF
        row[1] = NAN
    else:
        row[:] = 60.0
        row[0] = NAN
    if kind == "all beside a large row":      # in the same warp where rows share one
        z[bad - 1, 0] = z[bad + 1, 0] = 50.0
    out, status, _ = BL.call(moe, z, idx, None, seq, score, 0.3, 0.01)
    assert status == 0
    assert torch.isnan(out["loss"]).all()
    s = bad // seq if seq else 0
    assert torch.isnan(out["P"][s]).all()
    assert torch.isfinite(out["P"][[i for i in range(out["P"].shape[0]) if i != s]]).all()
    assert torch.isnan(out["dlogits"][bad]).all()
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[bad] = False
    assert torch.isfinite(out["dlogits"][rest]).all()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,n", [(2, 64), (24, 257), (300, 256), (300, 255), (2000, 264)])
def test_projection_forward(moe, act, out, T, n):
    """A NaN pre-activation stays one through every activation, and no other value is touched."""
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, 64), generator=g, device="cuda").bfloat16()
    W = torch.randn((n, 64), generator=g, device="cuda").bfloat16()
    b = torch.zeros(n, device="cuda")
    x[1, 3] = NAN
    b[5] = NAN
    cfg = moe.make_linear_config(T, 64, n, act=act, out_dtype=out)
    ws, y = moe.alloc_linear_workspace(cfg), torch.zeros((T, n), dtype=dt, device="cuda")
    moe.moe_linear_forward(cfg, x, W, b, None, None, y, ws)
    want = torch.zeros((T, n), dtype=torch.bool, device="cuda")
    want[1] = True
    want[:, 5] = True
    assert torch.equal(torch.isnan(y), want)
    assert torch.isfinite(y[~want]).all()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("n", [64, 63])
def test_projection_backward_through_relu(moe, out, n):
    """The gradient passes where the pre-activation is NaN, as it does in max(z, 0) by torch, and stops
    at negative values and zero."""
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    T = 70
    pre = torch.tensor([1.0, -1.0, 0.0, -0.0, NAN, INF, -INF], device="cuda").repeat(T * n // 7)[:T * n].view(T, n).to(dt)
    dy = (torch.arange(T * n, device="cuda") % 31 + 1.0).view(T, n).to(dt)
    cfg = moe.make_linear_config(T, 64, n, act="relu", out_dtype=out)
    ws, db = moe.alloc_linear_workspace(cfg), torch.zeros(n, device="cuda")
    moe.moe_linear_backward(cfg, None, None, pre, dy, None, None, db, ws)
    zero = torch.zeros((), dtype=dt, device="cuda")
    assert torch.equal(db, torch.where(pre <= 0, zero, dy).float().sum(0))
