"""The router's balance loss, its counts and its gradient against the float64 oracle, within the
oracle's derived bounds; and the gradient's way into the layer's backward pass."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from tests.conftest import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    ensure_built()
    import routing_shared_expert_gb300 as moe
    return moe


def config(moe, T, N, K, score="softmax"):
    return moe.make_config(T=T, d_model=64, N=N, K=K, d_expert=64, d_shared=0, shared_mode="none", score=score)


def batch(T, N, K, seed=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn((T, N), generator=g, device="cuda") * spread + torch.randn((1, N), generator=g, device="cuda")
    return z, torch.topk(z, K, dim=1).indices.to(torch.int32) if T else torch.empty((0, K), dtype=torch.int32, device="cuda")


def call(moe, z, idx, mask, L, score, cb, cz, gs=None, ws=None):
    T, N = z.shape
    K = idx.shape[1]
    cfg = config(moe, T, N, K, score)
    S = -(-T // (min(L, T) or T)) if T else 0
    out = {"counts": torch.full((S, N), -7, dtype=torch.int32, device="cuda"), "P": torch.full((S, N), 7.0, device="cuda"),
           "loss": torch.full((3,), 7.0, device="cuda"), "dlogits": torch.full((T, N), 7.0, device="cuda")}
    ws = moe.alloc_balance_loss_workspace(cfg, L) if ws is None else ws
    moe.moe_balance_loss(cfg, z, idx, mask, L, cb, cz, gs, out["counts"], out["P"], out["loss"], out["dlogits"], ws)
    return out, moe.moe_read_status(ws), ws


def check(moe, z, idx, mask=None, L=0, score="softmax", cb=0.3, cz=0.01, gs=None):
    out, status, ws = call(moe, z, idx, mask, L, score, cb, cz, gs)
    assert status == 0
    N, K = z.shape[1], idx.shape[1]
    ref = B.balance_loss(z, idx, mask, L, score, np.float32(cb).item(), np.float32(cz).item(), N, K,
                         1.0 if gs is None else float(gs))
    assert torch.equal(out["counts"].long(), ref["counts"])
    for k in ("P", "loss", "dlogits"):
        err, bound = (out[k].double().cpu() - ref[k].cpu()).abs(), ref[k + "_err"].cpu()
        assert torch.isfinite(out[k]).all(), k
        assert (err <= bound).all(), f"{k}: {float((err / bound.clamp(min=1e-300)).max()):.2f} times its bound"
    again, _, _ = call(moe, z, idx, mask, L, score, cb, cz, gs, ws)
    for k in out:
        assert torch.equal(out[k], again[k]), f"{k}: another call in the same workspace differs"
    return out


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 256, 8), (2, 3, 2), (17, 8, 2), (63, 60, 4), (64, 33, 3), (65, 64, 8),
                                   (200, 100, 5), (1000, 255, 8), (4097, 128, 6), (5000, 256, 8), (9000, 5, 1)])
def test_sizes(moe, score, T, N, K):
    check(moe, *batch(T, N, K), score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,L", [(100, 1), (100, 7), (100, 64), (100, 99), (100, 100), (100, 1000), (3000, 128),
                                 (3001, 500), (20000, 3000), (40000, 33)])
def test_sequences(moe, score, T, L):
    check(moe, *batch(T, 24, 3), L=L, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks(moe, score):
    z, idx = batch(700, 40, 4)
    for L in (0, 100, 64):
        mask = torch.ones(700, dtype=torch.uint8, device="cuda")
        mask[::3] = 0
        mask[100:200] = 0            # a whole sequence of 100
        mask[650:] = 0
        check(moe, z, idx, mask, L, score)
        bad = z.clone()
        bad[mask == 0] = float("nan")
        where = idx.clone()
        where[mask == 0] = -1
        a, b = check(moe, bad, where, mask, L, score), check(moe, z, idx, mask, L, score)
        for k in a:
            assert torch.equal(a[k], b[k]), "what a masked token holds has an effect"
        check(moe, z, idx, mask.bool(), L, score)
        out = check(moe, z, idx, torch.zeros_like(mask), L, score)
        for k in out:
            assert (out[k] == 0).all(), k


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(moe, score):
    z, idx = batch(300, 32, 4, spread=30.0)
    check(moe, z, idx, score=score)
    check(moe, z - 300.0, idx, score=score)      # every sigmoid underflows in fp32
    check(moe, z + 300.0, idx, score=score)
    z[:, 5] = -float("inf")                      # an expert switched off
    z[7] = -float("inf")                         # a token with no logit left
    z[8, :31] = -float("inf")
    z[9] = torch.finfo(torch.float32).min
    z[9, 3] = 0.0
    check(moe, z, idx, score=score, cz=0.0)
    z[9] = 0.0
    check(moe, z, idx, score=score)


def test_balanced_and_collapsed_routers(moe):
    z, _ = batch(64, 8, 8)
    every = torch.arange(8, dtype=torch.int32, device="cuda").expand(64, 8).contiguous()
    for score in ("softmax", "sigmoid"):
        out = check(moe, z, every, score=score, cz=0.0)
        assert (out["dlogits"] == 0).all(), "every expert has the same share: no gradient"
        one = torch.zeros((64, 1), dtype=torch.int32, device="cuda")
        check(moe, z, one, score=score)
    z = torch.zeros((64, 8), device="cuda")
    out = check(moe, z, every[:, :1].contiguous(), cz=0.0)
    assert float(out["loss"][1]) == 1.0


def test_grad_scale_and_missing_outputs(moe):
    z, idx = batch(500, 60, 4)
    gs = torch.tensor([2.5], device="cuda")
    check(moe, z, idx, gs=gs)
    full = check(moe, z, idx, L=64)
    cfg = config(moe, 500, 60, 4)
    ws = moe.alloc_balance_loss_workspace(cfg, 64)
    for k in full:
        only = {n: torch.empty_like(full[n]) if n == k else None for n in full}
        moe.moe_balance_loss(cfg, z, idx, None, 64, 0.3, 0.01, None, only["counts"], only["P"], only["loss"],
                             only["dlogits"], ws)
        assert torch.equal(only[k], full[k])


def test_bad_indices_are_reported_and_empty_slots_are_not(moe):
    z, idx = batch(100, 16, 4)
    idx[3, 1] = -1
    out, status, _ = call(moe, z, idx, None, 0, "softmax", 0.3, 0.0)
    assert status == 0 and int(out["counts"].sum()) == 399
    check(moe, z, idx)
    for bad in (16, -2, 2 ** 31 - 1):
        idx[3, 1] = bad
        out, status, _ = call(moe, z, idx, None, 0, "softmax", 0.3, 0.0)
        assert status == -6 and int(out["counts"].sum()) == 399


def test_no_tokens(moe):
    z, idx = batch(0, 8, 2)
    out, status, _ = call(moe, z, idx, None, 0, "softmax", 0.3, 0.1)
    assert status == 0 and (out["loss"] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(moe, score):
    z, idx = batch(90, 12, 3)
    g = torch.Generator(device="cuda").manual_seed(8)
    u = torch.randn(z.shape, generator=g, device="cuda").double()
    out, _, _ = call(moe, z, idx, None, 32, score, 0.3, 0.01)
    args = (idx, None, 32, score, np.float32(0.3).item(), np.float32(0.01).item(), 12, 3)
    h = 1e-5
    hi, lo = (float(B.balance_loss(z.double() + s * h * u, *args)["loss"][0]) for s in (1, -1))
    bound = float((B.balance_loss(z, *args)["dlogits_err"] * u.abs()).sum()) + 1e-8
    assert abs((hi - lo) / (2 * h) - float((out["dlogits"].double() * u).sum())) < bound


def test_graph_replay_takes_new_logits(moe):
    z, idx = batch(2000, 64, 4)
    cfg = config(moe, 2000, 64, 4)
    ws = moe.alloc_balance_loss_workspace(cfg, 256)
    loss, dz = torch.empty(3, device="cuda"), torch.empty_like(z)

    def run():
        moe.moe_balance_loss(cfg, z, idx, None, 256, 0.3, 0.01, None, None, None, loss, dz, ws)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    z.copy_(batch(2000, 64, 4, seed=5)[0])
    graph.replay()
    a, b = loss.clone(), dz.clone()
    run()
    assert torch.equal(a, loss) and torch.equal(b, dz) and moe.moe_read_status(ws) == 0


@pytest.mark.parametrize("name", ["olmo", "dsv3"])
def test_gradient_reaches_the_router(moe, name):
    """The layer's backward pass with dlogits: dW_router gains dlogits^T x and dx gains
    dlogits W_router, within the backward pass's bar (its operands are rounded to bf16); without
    dlogits it is the plain entry point bit for bit."""
    import oracle as O
    from workloads import CONFIGS, make_inputs
    spec = CONFIGS[name].replace(T=256, d_model=256, N=32, K=4, d_expert=128, d_shared=128, num_ranks=1)
    inp = make_inputs(spec, "cuda")
    layer = moe.MoELayer(moe.config_from_spec(spec), inp, "cuda")
    layer.forward(inp["x"])
    g = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.randn((256, 256), generator=g, device="cuda") * 1e-2
    ws = moe.alloc_balance_loss_workspace(layer.cfg, 64)
    dz = torch.empty((256, 32), device="cuda")
    moe.moe_balance_loss(layer.cfg, layer.out["logits"], layer.out["topk_idx"], None, 64, 1.0, 1.0, None, None,
                         None, None, dz, ws)
    plain = {k: v.clone() for k, v in layer.backward(inp["x"], dy, router_grad=True).items()}
    aux = {k: v.clone() for k, v in layer.backward(inp["x"], dy, router_grad=True, dlogits=dz).items()}
    assert layer.backward_status() == 0
    cpu = {k: (v.cpu() if torch.is_tensor(v) else v) for k, v in inp.items()}
    ref = O.moe_backward(spec, cpu, dy.cpu().numpy(), router_grad=True, logits=layer.out["logits"].cpu().numpy())
    d = dz.double().cpu()
    for k, add in (("dW_router", d.t() @ cpu["x"].double()), ("dx", d @ cpu["W_router"].double())):
        want = torch.from_numpy(ref[k]) + add
        rms = float((aux[k].double().cpu() - want).square().mean().sqrt() / want.square().mean().sqrt())
        assert rms <= 1.5e-2, (k, rms)
        # the added part is not lost in the bar
        assert float(add.square().mean().sqrt() / want.square().mean().sqrt()) > (0.1 if k == "dW_router" else 0.0)
    for k in plain:
        if k not in ("dx", "dW_router"):
            assert torch.equal(plain[k], aux[k]), k
    moe.moe_layer_backward(layer.cfg_bwd, layer.w_bwd, inp["x"], layer.outputs, dy, layer.grads_c, layer.bwd_ws)
    for k in plain:
        assert torch.equal(plain[k], layer.grads[k]), k
