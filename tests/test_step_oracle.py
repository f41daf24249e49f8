"""The oracles of the operators around the block against differences and independent forms (CPU only)."""
import math

import pytest
import torch

from oracle import step_oracle as S

F64 = torch.float64


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("residual", [False, True])
def test_layernorm_gradients_against_differences(kind, residual):
    g = torch.Generator().manual_seed(1)
    x, r, u = (torch.randn((6, 9), generator=g, dtype=F64) for _ in range(3))
    w, b, uw = (torch.randn(9, generator=g, dtype=F64) for _ in range(3))
    dy, ds = (torch.randn((6, 9), generator=g, dtype=F64) for _ in range(2))
    eps = 1e-3

    def value(h, w, b):
        """From the definition, apart from the oracle."""
        c = h - h.mean(1, keepdim=True) if kind == "layer" else h
        y = c / (c.square().mean(1, keepdim=True) + eps).sqrt() * w + b
        return float((y * dy).sum() + ((h * ds).sum() if residual else 0))

    h = x + r if residual else x
    f = S.layernorm(x, r if residual else None, w, b, eps, kind, None, F64)
    y = (h - h.mean(1, keepdim=True) if kind == "layer" else h) * f["rstd"][0][:, None] * w + b
    assert (f["y"][0] - y).abs().max() < 1e-12
    o = S.layernorm_backward(h, w, f["mean"][0], f["rstd"][0], dy, ds if residual else None, kind, F64)
    s = 1e-6
    for got, hi, lo in ((float((o["dx"][0] * u).sum()), (h + s * u, w, b), (h - s * u, w, b)),
                        (float((o["dweight"][0] * uw).sum()), (h, w + s * uw, b), (h, w - s * uw, b)),
                        (float((o["dbias"][0] * uw).sum()), (h, w, b + s * uw), (h, w, b - s * uw))):
        assert abs((value(*hi) - value(*lo)) / (2 * s) - got) < 1e-7 * (1 + abs(got))


def test_embedding_is_linear_and_its_gradient_the_transpose():
    g = torch.Generator().manual_seed(2)
    V, d = 7, 5
    ids = torch.tensor([3, -1, 3, 0, 6, 9, 3])      # a token past the table counts nowhere
    table, dout = torch.randn((V, d), generator=g, dtype=F64), torch.randn((len(ids), d), generator=g, dtype=F64)
    out, bound = S.embedding(ids, table, 1.5, torch.float32)
    assert torch.equal(out[[1, 5]], torch.zeros(2, d, dtype=F64)) and torch.equal(bound[1], out[1])
    assert torch.allclose(out[0], 1.5 * table[3])
    dt, _ = S.embedding_backward(ids, dout, 1.5, V, torch.float32)
    assert abs(float((out * dout).sum() - (dt * table).sum())) < 1e-12
    assert torch.equal(dt[1], torch.zeros(d, dtype=F64))
    held = torch.randn((V, d), generator=g, dtype=F64)
    assert torch.allclose(S.embedding_backward(ids, dout, 1.5, V, torch.float32, held)[0], held + dt)


def test_clipping():
    grads = [torch.full((3,), 2.0), torch.full((2, 2), 1.0, dtype=torch.bfloat16)]
    norm, coef, _, _ = S.grad_norm(grads, 2.0)
    assert norm == 4.0 and abs(coef - 2.0 / 4.000001) < 1e-15
    assert S.grad_norm(grads, 8.0)[1] == 1.0 and S.grad_norm(grads, math.inf)[1] == 1.0
    assert S.grad_norm([], 1.0)[:2] == (0.0, 1.0)
    clipped = S.clip(grads, 2.0)
    total = math.sqrt(sum(float((v ** 2).sum()) for v, _ in clipped))
    assert abs(total - 2.0) < 1e-6
