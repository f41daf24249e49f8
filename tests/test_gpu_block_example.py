"""The block of examples/train_block.py: its operators together, against a float64 restatement of
the whole block for the outputs and by differences for the gradients, and a few training steps."""
import importlib.util
import os

import pytest
import torch

from oracle import block_oracle as B
from tests.conftest import ROOT, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    ensure_built()
    path = os.path.join(ROOT, "examples", "train_block.py")
    spec = importlib.util.spec_from_file_location("train_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def make(example, T=300):
    from workloads import CONFIGS
    spec = CONFIGS["olmo"].replace(T=T, d_model=256, d_expert=128, d_shared=128, N=16, K=2, alpha=2.0)
    return example.Block(spec, seq_len=100, p=0.25)


def test_operators_together(example):
    b = make(example)
    out = b.forward()
    x, W = b.x, b.W_o
    ref_h, _, bound, _ = B.linear(x, W, b.b_o, x, "none", torch.bfloat16)
    assert ((b.h.double() - ref_h).abs() <= bound).all()
    ref, bound = B.dropout(b.layer.out["y"], b.h, 0.25, 0, 0, torch.float32)
    assert ((out.double() - ref).abs() <= bound).all()
    r = B.balance_loss(b.layer.out["logits"], b.layer.out["topk_idx"], None, 100, "softmax", b.coef_balance,
                       b.coef_z, b.spec.N, b.spec.K)
    # the coefficients reach the kernel as fp32: half a step of each, relative
    err = (b.bal.double().cpu() - r["loss"]).abs()
    assert (err <= r["loss_err"] + 2 * B.EPS32 * r["loss"].abs()).all()
    dout = torch.randn(out.shape, device="cuda")
    g = b.backward(dout)
    keep = B.keep_mask(*out.shape, 0.25, 0, 0).cuda()
    assert torch.equal(b.dy != 0, keep & (dout != 0))
    # the projection's gradients for the dh the block formed
    dh = (dout + b.layer.grads["dx"]).bfloat16()
    want = B.linear_backward(x, W, None, dh, "none", torch.bfloat16, torch.bfloat16, torch.float32)
    for name, got in (("dx", b.dx), ("dW", g["W_o"]), ("dbias", g["b_o"])):
        assert ((got.double() - want[name][0]).abs() <= want[name][1]).all(), name
    assert b.status() == 0


def test_training_lowers_the_loss_and_changes_the_mask(example):
    b = make(example)
    first = b.forward().clone()
    mask0 = (b.out != b.h.float())
    losses = [float(b.step()[0]) for _ in range(8)]
    assert losses[-1] < losses[0], losses
    b.forward()
    assert not torch.equal(mask0, b.out != b.h.float())
    assert torch.isfinite(b.out).all() and first.shape == b.out.shape
    assert b.status() == 0


def test_a_step_repeats_bit_for_bit(example):
    a, b = make(example), make(example)
    for _ in range(2):
        la, lb = a.step(), b.step()
        assert torch.equal(la[0], lb[0]) and torch.equal(la[1], lb[1])
    assert torch.equal(a.W_o, b.W_o) and torch.equal(a.weights["W_router"], b.weights["W_router"])
