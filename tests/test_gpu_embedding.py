"""Token embedding and the gradient of its table: within the oracle's rounding bounds on every type, size and
distribution of tokens, with nothing written outside the results."""
import math

import pytest
import torch

from oracle import step_oracle as S
from tests.conftest import ensure_built
from tests.test_gpu_layernorm import DT, Rows, gen, near, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    ensure_built()
    import routing_shared_expert_gb300 as moe
    return moe


def tokens(g, T, V, spread="zipf", dtype=torch.int64):
    """Token numbers: about 1 / rank, all the same, all apart, or in the table's order."""
    if spread == "same":
        ids = torch.full((T,), V // 2, device="cuda")
    elif spread == "sorted":
        ids = torch.arange(T, device="cuda") * V // max(T, 1)
    elif spread == "runs":        # lengths about those that the sums are cut at
        n = torch.tensor([64, 128, 63, 65, 8, 72, 1, 192, 127, 129, 32, 56, 2000, 7, 256, 640])
        n = n.repeat(T // int(n.sum()) + 1)
        ids = torch.repeat_interleave(torch.arange(len(n)) % V, n)[:T].cuda()
        ids = ids[torch.randperm(T, generator=g, device="cuda")]
    elif spread == "none":
        ids = torch.full((T,), -1, device="cuda")
    elif spread == "uniform":
        ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    else:
        u = torch.rand((T,), generator=g, device="cuda", dtype=torch.float64)
        rank = (torch.exp(u * math.log(V + 1.0)).long() - 1).clamp(0, V - 1)
        ids = torch.randperm(V, generator=g, device="cuda")[rank]
        ids = torch.where(torch.rand((T,), generator=g, device="cuda") < 0.1, torch.full_like(ids, -1), ids)
    return ids.to(dtype)


def check(moe, T, V, d, spread="zipf", table="f32", out="bf16", scale=1.0, ids_dtype=torch.int64, ldt=0, ldo=0, off=0,
          accumulate=False):
    g = gen(T * 7 + V + d)
    ids = tokens(g, T, V, spread, ids_dtype)
    ws = moe.alloc_embedding_workspace(T, V, d)
    ws[256:] = 0xFF
    W = Rows(V, d, DT[table], ldt, off, rand(g, V, d))
    Y = Rows(T, d, DT[out], ldo, off)
    moe.moe_embedding_forward(ids, W.v, scale, Y.v, ws)
    near(Y.v, S.embedding(ids, W.v, scale, DT[out]), "out")
    assert Y.untouched_around()
    dY = Rows(T, d, DT[out], ldo, off, rand(g, T, d))
    dY.v[ids < 0] = math.nan            # not looked at
    dW = Rows(V, d, DT[table], ldt, off, rand(g, V, d) if accumulate else None)
    held = dW.v.clone() if accumulate else None
    moe.moe_embedding_backward(ids, dY.v, scale, dW.v, ws, accumulate=accumulate)
    near(dW.v, S.embedding_backward(ids, dY.v, scale, V, DT[table], held), "dtable")
    assert dW.untouched_around() and moe.moe_read_status(ws) == 0
    # the same bits again, on the workspace as the first call left it
    again = Rows(V, d, DT[table], ldt, off, held)
    moe.moe_embedding_backward(ids, dY.v, scale, again.v, ws, accumulate=accumulate)
    assert torch.equal(again.v, dW.v)


SIZES = [(1, 1, 1), (1, 7, 8), (2, 3, 5), (5, 100, 64), (31, 10, 33), (32, 1000, 256), (33, 1000, 257), (300, 1000, 256),
         (257, 4097, 96), (1000, 50, 40), (2049, 300, 130), (4095, 5000, 64), (4096, 70000, 24), (4097, 5000, 64),
         (8192, 100, 72), (9001, 66000, 40), (20000, 3001, 136), (40000, 131073, 16), (70001, 513, 8), (131072, 2, 32),
         (150000, 200000, 9), (513, 300, 2051), (6000, 900, 2560),
         (5001, 300, 8), (4999, 300, 128), (7000, 40, 136), (9000, 3000, 256), (4100, 600000, 8), (4096, 300, 16),
         (5003, 70, 1), (4999, 300, 33), (6001, 200, 255)]


@pytest.mark.parametrize("T,V,d", SIZES)
def test_sizes(moe, T, V, d):
    check(moe, T, V, d)
    check(moe, T, V, d, table="bf16", out="f32", scale=math.sqrt(d), ids_dtype=torch.int32)


@pytest.mark.parametrize("spread", ["same", "sorted", "none", "uniform"])
@pytest.mark.parametrize("T,V,d", [(700, 97, 64), (5000, 400, 72), (5000, 70000, 33), (33000, 1000, 48)])
def test_spreads(moe, spread, T, V, d):
    check(moe, T, V, d, spread)
    check(moe, T, V, d, spread, accumulate=True)


@pytest.mark.parametrize("table", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("accumulate", [False, True])
def test_types(moe, table, out, ids, accumulate):
    for T, V, d in ((200, 90, 264), (200, 90, 131), (6000, 500, 264), (6000, 500, 131)):
        check(moe, T, V, d, "zipf", table, out, -0.75, ids, accumulate=accumulate)


@pytest.mark.parametrize("ldt,ldo,off", [(272, 264, 0), (257, 259, 0), (0, 0, 1), (0, 264, 3), (300, 0, 8)])
@pytest.mark.parametrize("d", [256, 250])
@pytest.mark.parametrize("T", [333, 7000])
def test_strides_and_offsets(moe, ldt, ldo, off, d, T):
    check(moe, T, 77, d, ldt=ldt, ldo=ldo, off=off)
    check(moe, T, 77, d, table="bf16", out="f32", ldt=ldt, ldo=ldo, off=off, accumulate=True)


@pytest.mark.parametrize("T", [9, 3000, 9000])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_tokens_outside_the_table(moe, T, dtype):
    """They read and write nothing, and show in the status word."""
    V, d = 60, 40
    g = gen(T)
    good = tokens(g, T, V, "uniform", dtype)
    for bad in (V, -2, torch.iinfo(dtype).max, torch.iinfo(dtype).min):
        ids = good.clone()
        ids[T // 2] = bad
        ws = moe.alloc_embedding_workspace(T, V, d)
        table, out = rand(g, V, d), torch.full((T, d), 7.0, device="cuda")
        moe.moe_embedding_forward(ids, table, 2.0, out, ws)
        near(out, S.embedding(ids, table, 2.0, torch.float32), "out")
        assert not out[T // 2].any() and moe.moe_read_status(ws) == -6
        dout, dt = rand(g, T, d), torch.full((V, d), 7.0, device="cuda")
        dout[T // 2] = math.nan
        moe.moe_embedding_backward(ids, dout, 2.0, dt, ws)
        near(dt, S.embedding_backward(ids, dout, 2.0, V, torch.float32), "dtable")
        assert moe.moe_read_status(ws) == -6 and moe.moe_read_status(ws) == 0
    # -1 is no token, and leaves nothing
    ids = good.clone()
    ids[::3] = -1
    moe.moe_embedding_backward(ids, dout, 2.0, dt, ws)
    assert moe.moe_read_status(ws) == 0


def test_infinities_and_nan_stay_with_their_tokens(moe):
    g = gen(3)
    for T in (500, 9000):
        V, d = 50, 64
        ids = tokens(g, T, V, "uniform")
        ids[7] = 11
        dout = rand(g, T, d)
        dout[7, 5] = math.nan
        dt, ws = torch.empty((V, d), device="cuda"), moe.alloc_embedding_workspace(T, V, d)
        moe.moe_embedding_backward(ids, dout, 1.0, dt, ws)
        bad = torch.isnan(dt)
        assert bad[11, 5] and int(bad.sum()) == 1
        table = rand(g, V, d)
        table[11] = math.inf
        out = torch.empty((T, d), device="cuda")
        moe.moe_embedding_forward(ids, table, 1.0, out, ws)
        assert torch.equal(torch.isinf(out).all(1), ids == 11) and torch.equal(torch.isinf(out).any(1), ids == 11)


def test_gradient_against_differences(moe):
    """out is linear in the table: its difference along a direction equals the gradient's product with it up to
    the roundings of the two results."""
    g = gen(4)
    for T, V, d in ((300, 40, 70), (6000, 700, 33)):
        ids = tokens(g, T, V)
        u, dout = rand(g, V, d), rand(g, T, d)
        out, dt, ws = torch.empty((T, d), device="cuda"), torch.empty((V, d), device="cuda"), moe.alloc_embedding_workspace(T, V, d)
        moe.moe_embedding_forward(ids, u, 1.25, out, ws)
        moe.moe_embedding_backward(ids, dout, 1.25, dt, ws)
        slope = float((out.double() * dout.double()).sum())
        bound = float((S.embedding(ids, u, 1.25, torch.float32)[1] * dout.double().abs()).sum())
        bound += float((S.embedding_backward(ids, dout, 1.25, V, torch.float32)[1] * u.double().abs()).sum())
        assert abs(slope - float((dt.double() * u.double()).sum())) <= bound


def test_token_numbers_of_any_shape(moe):
    g = gen(5)
    ids = tokens(g, 60, 30).view(3, 4, 5)
    table = rand(g, 30, 16)
    out, flat = torch.empty((3, 4, 5, 16), device="cuda"), torch.empty((60, 16), device="cuda")
    ws = moe.alloc_embedding_workspace(60, 30, 16)
    moe.moe_embedding_forward(ids, table, 1.0, out, ws)
    moe.moe_embedding_forward(ids, table, 1.0, flat, ws)
    assert torch.equal(out.view(60, 16), flat)
    a, b = torch.empty_like(table), torch.empty_like(table)
    moe.moe_embedding_backward(ids, out, 1.0, a, ws)
    moe.moe_embedding_backward(ids.view(-1), flat, 1.0, b, ws)
    assert torch.equal(a, b)


def test_no_tokens(moe):
    ids, none = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty((0, 8), device="cuda")
    ws = moe.alloc_embedding_workspace(0, 5, 8)
    moe.moe_embedding_forward(ids, torch.ones((5, 8), device="cuda"), 1.0, none, ws)
    dt = torch.ones((5, 8), device="cuda")
    moe.moe_embedding_backward(ids, none, 1.0, dt, ws, accumulate=True)
    assert (dt == 1).all()
    moe.moe_embedding_backward(ids, none, 1.0, dt, ws)
    assert not dt.any()


@pytest.mark.parametrize("T", [400, 12000])
def test_in_a_graph_on_another_stream_with_new_tokens(moe, T):
    g = gen(6)
    V, d = 300, 128
    ids, dout = tokens(g, T, V), rand(g, T, d)
    dt, ws = torch.empty((V, d), device="cuda"), moe.alloc_embedding_workspace(T, V, d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        moe.moe_embedding_backward(ids, dout, 1.0, dt, ws)
        with torch.cuda.graph(graph, stream=side):
            moe.moe_embedding_backward(ids, dout, 1.0, dt, ws)
    torch.cuda.synchronize()
    for spread in ("same", "zipf", "none", "sorted", "uniform"):
        ids.copy_(tokens(g, T, V, spread))
        dt.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        near(dt, S.embedding_backward(ids, dout, 1.0, V, torch.float32), spread)


def test_one_workspace_for_calls_of_different_sizes(moe):
    """A workspace of the largest call serves smaller ones, whatever an earlier call left in it."""
    g = gen(7)
    ws = moe.alloc_embedding_workspace(30000, 2000, 64)
    for T, V, d in ((30000, 2000, 64), (100, 2000, 64), (9000, 500, 40), (30000, 100, 64), (4500, 2000, 8)):
        if moe.moe_embedding_workspace_size(T, V, d) > ws.numel():
            continue
        ids, dout, dt = tokens(g, T, V), rand(g, T, d), torch.empty((V, d), device="cuda")
        moe.moe_embedding_backward(ids, dout, 1.0, dt, ws)
        near(dt, S.embedding_backward(ids, dout, 1.0, V, torch.float32), (T, V, d))


@pytest.mark.parametrize("spread", ["zipf", "same", "sorted", "uniform", "runs"])
@pytest.mark.parametrize("T,V,d", [(640, 300, 64), (4096, 900, 64), (4097, 900, 131), (16384, 500, 256), (16385, 500, 256),
                                   (19456, 3000, 450), (12970, 300, 768), (12971, 300, 767), (39001, 1000, 48)])
def test_about_the_length_of_the_chunks(moe, T, V, d, spread):
    """Both lengths of what a warp adds up, on either side of where they change; nothing is written behind the
    workspace's end."""
    g = gen(T + d)
    n = moe.moe_embedding_workspace_size(T, V, d)
    ws = torch.full((n + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    ws[:256] = moe.alloc_embedding_workspace(T, V, d)[:256]
    ids, dout = tokens(g, T, V, spread), rand(g, T, d).bfloat16()
    dt = torch.empty((V, d), device="cuda")
    moe.moe_embedding_backward(ids, dout, 0.5, dt, ws[:n])
    near(dt, S.embedding_backward(ids, dout, 0.5, V, torch.float32), "dtable")
    assert moe.moe_read_status(ws) == 0 and bool((ws[n:] == 0xA5).all())


def test_a_workspace_serves_fewer_tokens(moe):
    g = gen(11)
    V, d = 700, 520
    ws = moe.alloc_embedding_workspace(140000, V, d)
    for T in (140000, 131104, 131072, 12971, 12970, 4096, 2048, 513, 1):
        ids, dout, dt = tokens(g, T, V), rand(g, T, d).bfloat16(), torch.empty((V, d), device="cuda")
        moe.moe_embedding_backward(ids, dout, 1.0, dt, ws)
        near(dt, S.embedding_backward(ids, dout, 1.0, V, torch.float32), T)


def test_offsets_past_32_bits(moe):
    """A table and a gradient of more than 2^31 elements, tokens at both ends."""
    V, d, T = 70000, 32768, 96
    table = torch.empty((V, d), dtype=torch.bfloat16, device="cuda")
    table.fill_(1.0)
    ids = torch.tensor([0, V - 1, V // 2, V - 2] * (T // 4), device="cuda")
    table[ids] = rand(gen(9), T, d).bfloat16()
    out, ws = torch.empty((T, d), dtype=torch.bfloat16, device="cuda"), moe.alloc_embedding_workspace(T, V, d)
    moe.moe_embedding_forward(ids, table, 1.0, out, ws)
    assert torch.equal(out, table[ids])
    table.fill_(7.0)
    moe.moe_embedding_backward(ids, out, 1.0, table, ws)
    rows, inv = torch.unique(ids, return_inverse=True)
    small, bound = S.embedding_backward(inv, out, 1.0, len(rows), torch.bfloat16)
    near(table[rows], (small, bound), "rows")
    table[rows] = 0
    for a in range(0, V, 10000):
        assert not table[a:a + 10000].any()
