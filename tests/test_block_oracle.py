"""The oracles of the block operators against published values and differences (CPU only)."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B


def test_philox_known_answers():
    """The published known answers of Philox4x32-10 (zero, all-ones, and digits of pi)."""
    def words(c, k):
        counter, offset = c[0] | c[1] << 32, c[2] | c[3] << 32
        return [int(w) for w in B.philox([counter], k[0] | k[1] << 32, offset)[0]]

    assert words((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert words((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert words((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_keep_rate_is_one_minus_p():
    for p in (0.1, 0.5):
        keep = B.keep_mask(1000, 1000, p, 12345, 678).double().mean().item()
        # five standard deviations of a million draws
        assert abs(keep - (1 - p)) < 5 * (p * (1 - p) / 1e6) ** 0.5


@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_projection_gradients_against_differences(kind):
    g = torch.Generator().manual_seed(3)
    x, W, b = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((7, 5), (6, 5), (6,)))
    dy = torch.randn((7, 6), generator=g, dtype=torch.float64)

    def loss(x, W, b):
        return float((B.act(x @ W.t() + b, kind) * dy).sum())

    pre = x @ W.t() + b
    out = B.linear_backward(x, W, pre, dy, kind, torch.float32, torch.float32, torch.float32)
    h = 1e-6
    for i, name in enumerate(("dx", "dW", "dbias")):
        u = torch.randn((x, W, b)[i].shape, generator=g, dtype=torch.float64)
        hi, lo = [v.clone() for v in (x, W, b)], [v.clone() for v in (x, W, b)]
        hi[i] += h * u
        lo[i] -= h * u
        slope = (loss(*hi) - loss(*lo)) / (2 * h)
        assert abs(slope - float((out[name][0] * u).sum())) < 1e-6 * (1 + abs(slope))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("seq_len", [0, 5])
def test_balance_gradient_against_differences(score, seq_len):
    """With the counts held fixed (the selection does not move), the loss's differences."""
    g = torch.Generator().manual_seed(4)
    T, N, K = 13, 6, 2
    z = torch.randn((T, N), generator=g, dtype=torch.float64)
    idx = torch.topk(z, K, 1).indices.int()
    mask = torch.ones(T, dtype=torch.uint8)
    mask[[3, 12]] = 0
    args = (idx, mask, seq_len, score, 0.3, 0.02, N, K)
    got = B.balance_loss(z, *args)
    u = torch.randn((T, N), generator=g, dtype=torch.float64)
    h = 1e-6
    hi, lo = (float(B.balance_loss(z + s * h * u, *args)["loss"][0]) for s in (1, -1))
    assert abs((hi - lo) / (2 * h) - float((got["dlogits"] * u).sum())) < 1e-8
    assert torch.equal(got["dlogits"][3], torch.zeros(N, dtype=torch.float64))


def test_balance_loss_agrees_with_the_statistic():
    """One sequence without a mask: L of Eq. 30 as the layer oracle computes it."""
    import oracle as O
    g = torch.Generator().manual_seed(5)
    T, N, K = 50, 8, 2
    z = torch.randn((T, N), generator=g, dtype=torch.float64)
    idx = torch.topk(z, K, 1).indices.int()
    got = B.balance_loss(z, idx, None, 0, "softmax", 1.0, 0.0, N, K)
    _, P, L = O.lbl_statistics(torch.softmax(z, 1).numpy(), idx.numpy(), N)
    assert abs(float(got["loss"][1]) - L) < 1e-12
    assert np.abs(got["P"][0].numpy() - P).max() < 1e-14
