"""A matrix of one row has no row stride to speak of: whatever the configuration says of it, the call
is the dense one bit for bit."""
import pytest
import torch

from tests import test_gpu_linear as L
from tests.conftest import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    ensure_built()
    import routing_shared_expert_gb300 as moe
    return moe


# x, the residual, y and dy are one row for one token, W for one feature
@pytest.mark.parametrize("T,n_in,n_out,which", [(1, 64, 32, ("ldx", "ldr", "ldy")), (1, 4096, 16, ("ldx", "ldr", "ldy")),
                                                (8, 64, 1, ("ldw",)), (2, 1024, 1, ("ldw",)), (1, 72, 1, ("ldx", "ldw", "ldr", "ldy"))])
@pytest.mark.parametrize("ld", [4097, 1 << 39])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_any_stride_of_a_single_row(moe, T, n_in, n_out, which, ld, out):
    g = torch.Generator(device="cuda").manual_seed(1)
    dt = L.DT[out]
    x, W = L.rows(g, T, n_in, torch.bfloat16), L.rows(g, n_out, n_in, torch.bfloat16)
    r, dy = L.rows(g, T, n_out, dt), L.rows(g, T, n_out, dt)
    results = []
    for strides in ({}, {k: ld for k in which}):
        cfg = moe.make_linear_config(T, n_in, n_out, out_dtype=out, **strides)
        ws = moe.alloc_linear_workspace(cfg)
        y, dx, dW, db = (torch.full(s, 7.0, dtype=d, device="cuda") for s, d in
                         (((T, n_out), dt), ((T, n_in), torch.bfloat16), ((n_out, n_in), torch.bfloat16),
                          ((n_out,), torch.float32)))
        moe.moe_linear_forward(cfg, x, W, None, r, None, y, ws)
        moe.moe_linear_backward(cfg, x, W, None, dy, dx, dW, db, ws)
        assert moe.moe_read_status(ws) == 0
        results.append((y, dx, dW, db))
    for a, b in zip(*results):
        assert torch.equal(a, b)
