"""The block's operators past the sizes of the other tests: element offsets beyond 2^31, long
batches of the balance loss, and the share of a logit gradient in the layer's backward pass."""
import pytest
import torch

from oracle import block_oracle as B
from tests import test_gpu_balance_loss as BL
from tests import test_gpu_linear as L
from tests.conftest import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    ensure_built()
    import routing_shared_expert_gb300 as moe
    return moe


def test_projection_rows_past_32_bits(moe):
    """x (by its stride), the residual, pre, y and dy have over 2^31 elements."""
    T, i, o = 262144 + 700, 64, 8192
    assert T * o > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty((T, o), dtype=torch.bfloat16, device="cuda")[:, :i]
    x.copy_(torch.randn((T, i), generator=g, device="cuda"))
    W = L.rows(g, o, i, torch.bfloat16, std=i ** -0.5)
    b = torch.randn(o, generator=g, device="cuda")
    r = torch.randn((T, o), generator=g, device="cuda", dtype=torch.bfloat16)
    y, pre = torch.empty_like(r), torch.empty_like(r)
    cfg = moe.make_linear_config(T, i, o, act="silu", ldx=o, dw_dtype="f32")
    ws = moe.alloc_linear_workspace(cfg)
    moe.moe_linear_forward(cfg, x, W, b, r, pre, y, ws)
    spots = [slice(0, 300), slice(262144 - 150, 262144 + 150), slice(T - 300, T)]
    for s in spots:
        ref_y, ref_z, by, bz = B.linear(x[s], W, b, r[s], "silu", torch.bfloat16)
        L.within("y", y[s], ref_y, by)
        L.within("pre", pre[s], ref_z, bz)
    dx, dW, db = torch.empty((T, i), dtype=torch.bfloat16, device="cuda"), torch.empty((o, i), device="cuda"), \
        torch.empty(o, device="cuda")
    dy = r
    moe.moe_linear_backward(cfg, x, W, pre, dy, dx, dW, db, ws)
    assert moe.moe_read_status(ws) == 0
    total = {"dW": [0, 0], "dbias": [0, 0]}
    for t0 in range(0, T, 32768):
        s = slice(t0, min(T, t0 + 32768))
        ref = B.linear_backward(x[s], W, pre[s], dy[s], "silu", torch.bfloat16, torch.bfloat16, torch.float32)
        L.within("dx", dx[s], *ref["dx"])
        for k in total:
            # a part's bound grows with its 32768 terms; in the whole sum every product passes
            # T additions: T / 32768 times the parts' bounds
            total[k][0] = total[k][0] + ref[k][0]
            total[k][1] = total[k][1] + ref[k][1]
    for k, got in (("dW", dW), ("dbias", db)):
        value, bound = total[k]
        L.within(k, got, value, bound * (T / 32768 + 1))


@pytest.mark.parametrize("n_in", [8200, 8193])
def test_projection_weights_past_32_bits(moe, n_in):
    """One token through weights of over 2^31 elements, aligned rows and unaligned ones."""
    o = 262200
    assert o * n_in > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(4)
    x = L.rows(g, 1, n_in, torch.bfloat16)
    W = torch.randn((o, n_in), generator=g, device="cuda", dtype=torch.bfloat16)
    y = torch.empty((1, o), device="cuda")
    cfg = moe.make_linear_config(1, n_in, o, out_dtype="f32")
    ws = moe.alloc_linear_workspace(cfg)
    moe.moe_linear_forward(cfg, x, W, None, None, None, y, ws)
    assert moe.moe_read_status(ws) == 0
    for s in (slice(0, 500), slice(130000, 130500), slice(2 ** 31 // n_in - 250, 2 ** 31 // n_in + 250), slice(o - 500, o)):
        ref, _, bound, _ = B.linear(x, W[s], None, None, "none", torch.float32)
        L.within("y", y[:, s], ref, bound)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,N,K,seq", [(131072, 256, 8, 4096), (100003, 128, 6, 5000), (70001, 60, 4, 0),
                                       (65536, 8, 2, 64)])
def test_balance_loss_of_long_batches(moe, score, T, N, K, seq):
    z, idx = BL.batch(T, N, K)
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    mask[::5] = 0
    mask[T // 2:T // 2 + 3 * max(seq, 100)] = 0
    BL.check(moe, z, idx, None, seq, score)
    BL.check(moe, z, idx, mask, seq, score)


def test_logit_gradient_alone_in_the_layer(moe):
    """With dy = 0 nothing comes through the coefficients: dx = dlogits W_router and dW_router =
    dlogits^T x, each within one rounding of dlogits to bf16 and the fp32 sums."""
    from workloads import CONFIGS, make_inputs
    spec = CONFIGS["dsv3"].replace(T=256, d_model=256, N=32, K=4, d_expert=128, d_shared=128, num_ranks=1)
    inp = make_inputs(spec, "cuda")
    layer = moe.MoELayer(moe.config_from_spec(spec), inp, "cuda")
    layer.forward(inp["x"])
    dz = torch.randn((256, 32), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    dy = torch.zeros((256, 256), device="cuda")
    got = layer.backward(inp["x"], dy, router_grad=True, dlogits=dz)
    assert layer.backward_status() == 0
    d, W, x = dz.double(), inp["W_router"].double(), inp["x"].double()
    for k, a, b, n in (("dx", d, W, 32), ("dW_router", d.t(), x, 256)):
        rel = B.half_step(torch.bfloat16) + (n + 8) * 2.0 ** -23
        L.within(k, got[k], a @ b, rel * (a.abs() @ b.abs()))
    assert float(got["dx"].abs().max()) > 0 and (layer.backward(inp["x"], dy, router_grad=True)["dx"] == 0).all()
