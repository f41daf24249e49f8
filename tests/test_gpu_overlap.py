"""Chains of calls that each read what the one before wrote, over two buffers in turn and with
nothing between them, so that every launch begins under the previous one.  The weights are shifts
and the values whole numbers, so each result is known exactly: a value read before its launch had
the right to it stays in the chain to its end."""
import pytest
import torch

from tests.conftest import ensure_built

pytestmark = pytest.mark.gpu
STEPS = 48


@pytest.fixture(scope="module")
def moe():
    ensure_built()
    import routing_shared_expert_gb300 as moe
    return moe


def shift(n, by):
    """W with x W^T = x moved up by `by` places."""
    W = torch.zeros((n, n), dtype=torch.bfloat16, device="cuda")
    i = torch.arange(n, device="cuda")
    W[i, (i - by) % n] = 1.0
    return W


def numbers(T, n, dtype):
    return (torch.arange(T * n, device="cuda").view(T, n) * 7 % 251).to(dtype)


# one and a few tokens (a warp per weight row), few-token tiles, pair tiles; odd widths take
# unaligned loads or aligned copies
@pytest.mark.parametrize("n", [512, 513, 1001, 2048])
@pytest.mark.parametrize("T", [1, 2, 24, 300, 1100])
def test_forward_reads_the_previous_output(moe, T, n):
    cfg = moe.make_linear_config(T, n, n)
    ws, W = moe.alloc_linear_workspace(cfg), shift(n, 5)
    a = numbers(T, n, torch.bfloat16)
    start, b = a.clone(), torch.zeros_like(a)
    for turn in range(3):
        for _ in range(STEPS):
            moe.moe_linear_forward(cfg, a, W, None, None, None, b, ws)
            a, b = b, a
        assert torch.equal(a, start.roll(5 * STEPS * (turn + 1), 1))
    assert moe.moe_read_status(ws) == 0


@pytest.mark.parametrize("n", [512, 1001])
@pytest.mark.parametrize("T", [1, 24, 300])
def test_bias_and_residual_are_the_previous_output(moe, T, n):
    """y' = x W^T + y[0] + y: the bias is the first row of the output before, the residual all of it."""
    cfg = moe.make_linear_config(T, n, n, out_dtype="f32")
    ws, W = moe.alloc_linear_workspace(cfg), shift(n, 3)
    x = numbers(T, n, torch.bfloat16) % 4
    add = x.double().roll(3, 1)
    a, b = torch.zeros((T, n), device="cuda"), torch.zeros((T, n), device="cuda")
    want = torch.zeros((T, n), dtype=torch.float64, device="cuda")
    for _ in range(12):                 # below 2^24 at the end: exact
        moe.moe_linear_forward(cfg, x, W, a[0], a, None, b, ws)
        a, b = b, a
        want = add + want[0] + want
    assert float(want.max()) < 2 ** 24
    assert torch.equal(a.double(), want)


@pytest.mark.parametrize("n", [512, 1001])
@pytest.mark.parametrize("T", [1, 70, 300])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_backward_reads_the_previous_gradient(moe, T, n, out):
    """dx of one call is dy of the next; the pass that forms dz reads it and the pre-activations."""
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    cfg = moe.make_linear_config(T, n, n, act="relu", out_dtype=out, dx_dtype=out)
    ws, W = moe.alloc_linear_workspace(cfg), shift(n, -5)       # dz W moves up by five
    pre = torch.ones((T, n), dtype=dt, device="cuda")
    a = numbers(T, n, dt)
    start, b, db = a.clone(), torch.zeros_like(a), torch.zeros(n, device="cuda")
    x = torch.zeros((T, n), dtype=torch.bfloat16, device="cuda")
    for _ in range(STEPS):
        moe.moe_linear_backward(cfg, x, W, pre, a, b, None, db, ws)
        a, b = b, a
    assert torch.equal(a, start.roll(5 * STEPS, 1))
    # the last call's dy, summed over the tokens: whole numbers below 2^24
    assert torch.equal(db, start.roll(5 * (STEPS - 1), 1).float().sum(0))


@pytest.mark.parametrize("T,n", [(1, 512), (1, 513), (24, 512), (300, 512), (300, 1001)])
def test_forward_and_backward_in_turn(moe, T, n):
    """pre is rewritten by every forward call and read by the backward call behind it."""
    cfg = moe.make_linear_config(T, n, n, act="relu")
    ws, W = moe.alloc_linear_workspace(cfg), shift(n, 5)
    x = numbers(T, n, torch.bfloat16) - 125
    bufs = [torch.zeros_like(x) for _ in range(2)]
    y, dx, pre = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    dy = numbers(T, n, torch.bfloat16) % 64 + 1
    seen = []
    for i in range(8):
        moe.moe_linear_forward(cfg, x, W, None, None, pre, y, ws)
        moe.moe_linear_backward(cfg, x, W, pre, dy, dx, None, None, ws)
        # the next x: this one moved once more, so that pre changes sign in other places
        moe.moe_linear_forward(moe.make_linear_config(T, n, n), x, W, None, None, None, bufs[i % 2], ws)
        seen.append((x.clone(), dx.clone()))
        x = bufs[i % 2]
    for x, dx in seen:
        gate = (x.roll(5, 1) > 0).to(dy.dtype)
        assert torch.equal(dx, (dy * gate).roll(-5, 1))


@pytest.mark.parametrize("T,n", [(1, 512), (24, 512), (300, 512), (300, 511)])
def test_captured_beside_copies_and_another_stream(moe, T, n):
    """Captured: operands written by a copy node and by a call on a second stream that joins."""
    cfg, add = moe.make_linear_config(T, n, n), moe.make_linear_config(T, n, n)
    ws, ws2, W = moe.alloc_linear_workspace(cfg), moe.alloc_linear_workspace(cfg), shift(n, 5)
    src = numbers(T, n, torch.bfloat16) % 16
    x, a, b, y, z = (torch.zeros_like(src) for _ in range(5))
    side = torch.cuda.Stream()

    def work():
        main = torch.cuda.current_stream()
        x.copy_(src)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for _ in range(6):          # longer than what it joins
                moe.moe_linear_forward(cfg, x, W, None, None, None, a, ws2)
                moe.moe_linear_forward(cfg, a, W, None, None, None, b, ws2)
        moe.moe_linear_forward(cfg, x, W, None, None, None, y, ws)
        main.wait_stream(side)
        moe.moe_linear_forward(add, y, W, None, b, None, z, ws)     # reads both streams' outputs
        y.zero_()                                                   # and its operand is cleared behind it

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        work()
    torch.cuda.current_stream().wait_stream(warm)
    assert torch.equal(z, 2 * src.roll(10, 1))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for i in range(5):
        src.copy_(src.roll(1, 1))
        for t in (x, a, b, z):
            t.zero_()
        graph.replay()
        assert torch.equal(z, 2 * src.roll(10, 1)), i
        assert (y == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,N,seq", [(20000, 64, 0), (20000, 256, 2048), (600, 8, 100)])
def test_balance_loss_of_logits_rewritten_in_place(moe, score, T, N, seq):
    """The second launch of the loss begins under its first with logits that the call before it read
    as other values."""
    cfg = moe.make_config(T=T, d_model=64, N=N, K=2, d_expert=64, d_shared=0, shared_mode="none", score=score)
    ws = moe.alloc_balance_loss_workspace(cfg, seq)
    g = torch.Generator(device="cuda").manual_seed(0)
    base = torch.randn((T, N), generator=g, device="cuda")
    z, idx = torch.empty_like(base), torch.topk(base, 2, dim=1).indices.to(torch.int32)
    outs = [(torch.empty(3, device="cuda"), torch.empty_like(base)) for _ in range(12)]

    def turn(i, loss, dz):
        torch.mul(base, 1.0 - 0.125 * i, out=z)
        moe.moe_balance_loss(cfg, z, idx, None, seq, 0.3, 0.01, None, None, None, loss, dz, ws)

    for i, o in enumerate(outs):
        turn(i, *o)
    torch.cuda.synchronize()
    again = (torch.empty(3, device="cuda"), torch.empty_like(base))
    for i, o in enumerate(outs):
        turn(i, *again)
        torch.cuda.synchronize()
        assert torch.equal(o[0], again[0]) and torch.equal(o[1], again[1]), i
