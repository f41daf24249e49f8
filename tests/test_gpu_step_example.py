"""The embedded block of examples/train_block.py: token numbers, normalised halves and clipped gradients together
with the block's own operators, each against its float64 oracle on the operands that the run gave it."""
import importlib.util
import os

import pytest
import torch

from oracle import block_oracle as B
from oracle import step_oracle as S
from tests.conftest import ROOT, ensure_built
from tests.test_gpu_layernorm import near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    ensure_built()
    path = os.path.join(ROOT, "examples", "train_block.py")
    spec = importlib.util.spec_from_file_location("train_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def make(example, T=300, **kw):
    from workloads import CONFIGS
    spec = CONFIGS["olmo"].replace(T=T, d_model=256, d_expert=128, d_shared=128, N=16, K=2, alpha=2.0)
    return example.EmbeddedBlock(spec, seq_len=100, p=0.25, vocab=90, **kw)


def test_operators_together(example):
    b = make(example, max_norm=1e9)          # nothing to clip: the gradients stay as the operators wrote them
    out = b.forward()
    near(b.x, S.embedding(b.ids, b.table, b.scale, torch.bfloat16), "x")
    assert not b.x[-1].any()
    near(b.xn, S.layernorm(b.x, None, b.norm_1, None, b.eps, "rms", None, torch.bfloat16)["y"], "xn")
    ref_h, _, bound, _ = B.linear(b.xn, b.W_o, b.b_o, b.x, "none", torch.bfloat16)
    near(b.h, (ref_h, bound), "h")
    near(b.hn, S.layernorm(b.h, None, b.norm_2, None, b.eps, "rms", None, torch.bfloat16)["y"], "hn")
    near(out, B.dropout(b.layer.out["y"], b.h, 0.25, 0, 0, torch.float32), "out")
    dout = torch.randn(out.shape, device="cuda")
    g = b.backward(dout)
    assert float(b.grad_norm[1]) == 1.0
    want = S.layernorm_backward(b.h, b.norm_2, None, b.rstd_2, b.layer.grads["dx"], dout, "rms", torch.float32)
    near(b.dh32, want["dx"], "dh")
    near(g["norm_2"], want["dweight"], "dnorm_2")
    dh = b.dh32.bfloat16()
    want = B.linear_backward(b.xn, b.W_o, None, dh, "none", torch.bfloat16, torch.bfloat16, torch.float32)
    near(b.dx, want["dx"], "dxn")
    near(g["W_o"], want["dW"], "dW_o")
    want = S.layernorm_backward(b.x, b.norm_1, None, b.rstd_1, b.dx, dh, "rms", torch.bfloat16)
    near(b.de, want["dx"], "de")
    near(g["norm_1"], want["dweight"], "dnorm_1")
    near(g["table"], S.embedding_backward(b.ids, b.de, b.scale, 90, torch.float32), "dtable")
    norm, _, rel, _ = S.grad_norm(list(g.values()), 1e9)
    assert abs(float(b.grad_norm[0]) - norm) <= rel * norm
    assert b.status() == 0


def test_gradients_are_clipped_together(example):
    free, clipped = make(example, max_norm=1e9), make(example, max_norm=0.5)
    grads = []
    for b in (free, clipped):
        b.forward()
        grads.append(b.backward(torch.randn(b.out.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(3))))
    assert torch.equal(free.grad_norm[0], clipped.grad_norm[0]) and float(clipped.grad_norm[1]) < 1
    for name, want in zip(grads[0], S.clip(list(grads[0].values()), 0.5)):
        near(grads[1][name], want, name)
    total = float(sum((v.double() ** 2).sum() for v in grads[1].values()) ** 0.5)
    # 1e-6 in the factor's denominator, bf16 gradients rounded by half a step each at most
    assert abs(total - 0.5) <= 0.5 * 2.0 ** -8


def test_a_step_repeats_bit_for_bit(example):
    a, b = make(example), make(example)
    for _ in range(2):
        la, lb = a.step(), b.step()
        assert torch.equal(la[0], lb[0]) and torch.equal(la[1], lb[1])
    assert torch.equal(a.table, b.table) and torch.equal(a.W_o, b.W_o) and torch.equal(a.norm_1, b.norm_1)
    assert a.status() == 0 and torch.isfinite(a.table).all()


def test_it_runs_from_the_command_line(example):
    losses = example.main(["--steps", "3", "--tokens", "200", "--embedded"])
    assert len(losses) == 3 and all(loss == loss for loss in losses)
