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
