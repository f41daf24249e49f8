"""The dense projection and its gradients against the float64 oracle, elementwise within the
oracle's derived bounds: every activation and type, odd sizes, strides, and the forms chosen by
size and alignment."""
import pytest
import torch

from oracle import block_oracle as B
from tests.conftest import ensure_built

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CANARY = 7.0


@pytest.fixture(scope="module")
def moe():
    ensure_built()
    import routing_shared_expert_gb300 as moe
    return moe


def rows(g, T, n, dtype, std=1.0, ld=None, offset=0):
    """A [T][n] matrix of rows ``ld`` elements apart that starts ``offset`` elements into its
    buffer; what lies between the rows holds NaN."""
    ld = ld or n
    buf = torch.full((offset + T * ld + 16,), float("nan"), dtype=dtype, device="cuda")
    m = buf[offset:offset + T * ld].view(T, ld)[:, :n] if T else buf[:0].view(0, n)
    m.copy_(torch.randn((T, n), generator=g, device="cuda") * std)
    return m


def target(T, n, dtype, ld=None, offset=0):
    ld = ld or n
    buf = torch.full((offset + T * ld + 16,), CANARY, dtype=dtype, device="cuda")
    return buf[offset:offset + T * ld].view(T, ld)[:, :n] if T else buf[:0].view(0, n), buf


def only_written(view, buf):
    """Nothing outside the view changed."""
    mark = torch.zeros_like(buf, dtype=torch.bool)
    mark.as_strided(view.shape, view.stride(), view.storage_offset())[:] = True
    assert (buf[~mark] == CANARY).all(), "a value outside the output was written"


def within(name, got, ref, bound):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), name
    over = err > bound
    assert not over.any(), (f"{name}: {int(over.sum())} of {err.numel()} values outside their bound, worst "
                            f"{float((err / bound.clamp(min=1e-300)).max()):.2f} times")


def forward(moe, T, n_in, n_out, act="none", out="bf16", bias=True, residual=True, pre=True, ldx=0, ldw=0,
            ldr=0, ldy=0, off=0, in_place=False, ws=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    od = DT[out]
    x = rows(g, T, n_in, torch.bfloat16, ld=ldx, offset=off)
    W = rows(g, n_out, n_in, torch.bfloat16, std=n_in ** -0.5, ld=ldw, offset=off)
    b = torch.randn(n_out, generator=g, device="cuda") if bias else None
    y, ybuf = target(T, n_out, od, ldy, off)
    r = rows(g, T, n_out, od, ld=ldr, offset=off) if residual else None
    r0 = r.clone() if residual else None
    if in_place:
        y.copy_(r)
        r = y
    z, zbuf = target(T, n_out, od) if pre else (None, None)
    cfg = moe.make_linear_config(T, n_in, n_out, act=act, out_dtype=out, ldx=ldx, ldw=ldw, ldr=ldr, ldy=ldy)
    if ws is None:
        ws = moe.alloc_linear_workspace(cfg)
    moe.moe_linear_forward(cfg, x, W, b, r, z, y, ws)
    assert moe.moe_read_status(ws) == 0
    ref_y, ref_z, by, bz = B.linear(x, W, b, r0, act, od)
    within("y", y, ref_y, by)
    only_written(y, ybuf)
    if pre:
        within("pre", z, ref_z, bz)
        only_written(z, zbuf)
    return y, z


SIZES = [(1, 64, 64), (1, 2048, 2048), (2, 8, 1), (3, 72, 60), (7, 1000, 257), (16, 256, 130), (17, 512, 384),
         (33, 64, 1000), (64, 2048, 512), (127, 128, 128), (128, 320, 256), (129, 192, 264), (256, 1024, 640),
         (257, 2560, 512), (300, 64, 72), (1000, 200, 1407), (1237, 2048, 768), (2050, 136, 2056),
         (2700, 1024, 2048)]


@pytest.mark.parametrize("T,n_in,n_out", SIZES)
def test_forward_sizes(moe, T, n_in, n_out):
    for out in ("bf16", "f32"):
        forward(moe, T, n_in, n_out, act="silu", out=out)
        forward(moe, T, n_in, n_out, out=out, bias=False, residual=False, pre=False)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("T", [5, 600])
def test_forward_activations(moe, act, T):
    for out in ("bf16", "f32"):
        forward(moe, T, 256, 320, act=act, out=out, pre=False)
        forward(moe, T, 256, 320, act=act, out=out, residual=False)


@pytest.mark.parametrize("T,n_in,n_out", [(1, 1, 1), (1, 65, 33), (5, 131, 7), (40, 999, 301), (300, 65, 129),
                                          (513, 1001, 515)])
def test_forward_odd_features(moe, T, n_in, n_out):
    """Rows that do not start on 16-byte boundaries."""
    for out in ("bf16", "f32"):
        forward(moe, T, n_in, n_out, act="gelu", out=out)


@pytest.mark.parametrize("T,n_in,n_out", [(5200, 72, 1280), (5200, 72, 1100), (5200, 72, 1275), (20000, 64, 256)])
def test_forward_whole_and_narrow_tiles(moe, T, n_in, n_out):
    """A full round of tiles, then a partial one: 29 or 3 tiles on 76 pairs; 1100 and 1275 end inside
    the first and the second half of a tile."""
    for out in ("bf16", "f32"):
        forward(moe, T, n_in, n_out, act="gelu", out=out)
        forward(moe, T, n_in, n_out, out=out, bias=False, residual=False, pre=False)


@pytest.mark.parametrize("T", [1, 19, 130, 700])
def test_forward_strides_and_offsets(moe, T):
    forward(moe, T, 256, 192, act="silu", ldx=264, ldw=512, ldr=200, ldy=1024)      # aligned strides
    forward(moe, T, 256, 192, act="silu", ldx=257, ldw=259, ldr=193, ldy=195)       # unaligned ones
    forward(moe, T, 256, 192, out="f32", ldx=264, ldw=257, ldr=196, ldy=201)
    forward(moe, T, 256, 192, act="relu", off=1)                                    # bases off by one
    forward(moe, T, 256, 192, act="relu", out="f32", off=1)
    forward(moe, T, 256, 192, ldy=200, ldr=200, off=8)


@pytest.mark.parametrize("T,n_in,n_out", [(1, 512, 256), (40, 128, 321), (520, 256, 512), (520, 256, 321)])
def test_forward_residual_in_place(moe, T, n_in, n_out):
    for out in ("bf16", "f32"):
        forward(moe, T, n_in, n_out, act="gelu_tanh", out=out, in_place=True)


def test_forward_repeats_bit_for_bit_in_one_workspace(moe):
    """Different shapes through one workspace, in turn, twice: the same bits."""
    shapes = [(1, 2048, 512), (700, 512, 512), (24, 1024, 4096), (130, 999, 301)]
    size = max(moe.moe_linear_workspace_size(moe.make_linear_config(*s)) for s in shapes)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    first = [[t.clone() for t in forward(moe, *s, act="silu", ws=ws)] for s in shapes]
    again = [forward(moe, *s, act="silu", ws=ws) for s in shapes]
    for a, b in zip(first, again):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


def test_forward_no_tokens(moe):
    cfg = moe.make_linear_config(0, 64, 64)
    ws = moe.alloc_linear_workspace(cfg)
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    moe.moe_linear_forward(cfg, e, torch.zeros((64, 64), dtype=torch.bfloat16, device="cuda"), None, None, None, e, ws)
    assert moe.moe_read_status(ws) == 0


def test_nan_stays_in_its_row_and_column(moe):
    """A NaN in one token's input reaches that token alone, one in a weight row that feature."""
    for T in (3, 300):
        g = torch.Generator(device="cuda").manual_seed(1)
        x, W = rows(g, T, 136, torch.bfloat16), rows(g, 72, 136, torch.bfloat16)
        x[1, 135] = float("nan")
        W[5, 0] = float("inf")
        y = torch.zeros((T, 72), dtype=torch.bfloat16, device="cuda")
        cfg = moe.make_linear_config(T, 136, 72)
        moe.moe_linear_forward(cfg, x, W, None, None, None, y, moe.alloc_linear_workspace(cfg))
        bad = ~torch.isfinite(y)
        want = torch.zeros_like(bad)
        want[1, :] = True
        want[:, 5] = True
        assert torch.equal(bad, want)


def backward(moe, T, n_in, n_out, act="silu", out="bf16", dx_dtype="bf16", dw_dtype="bf16", ldx=0, ldw=0,
             ldy=0, off=0, want=("dx", "dW", "dbias"), seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    od = DT[out]
    x = rows(g, T, n_in, torch.bfloat16, ld=ldx, offset=off)
    W = rows(g, n_out, n_in, torch.bfloat16, std=n_in ** -0.5, ld=ldw, offset=off)
    pre = rows(g, T, n_out, od, offset=off) if act != "none" else None
    dy = rows(g, T, n_out, od, ld=ldy, offset=off)
    outs = {"dx": target(T, n_in, DT[dx_dtype], offset=off), "dW": target(n_out, n_in, DT[dw_dtype], offset=off),
            "dbias": target(1, n_out, torch.float32)}
    cfg = moe.make_linear_config(T, n_in, n_out, act=act, out_dtype=out, dx_dtype=dx_dtype, dw_dtype=dw_dtype,
                                 ldx=ldx, ldw=ldw, ldy=ldy)
    ws = moe.alloc_linear_workspace(cfg)
    v = {k: outs[k][0] if k in want else None for k in outs}
    moe.moe_linear_backward(cfg, x if v["dW"] is not None else None, W if v["dx"] is not None else None, pre, dy,
                            v["dx"], v["dW"], v["dbias"].view(-1) if v["dbias"] is not None else None, ws)
    assert moe.moe_read_status(ws) == 0
    ref = B.linear_backward(x, W, pre, dy, act, od, DT[dx_dtype], DT[dw_dtype])
    for k in want:
        within(k, v[k].view(ref[k][0].shape), *ref[k])
    for k in outs:
        if k in want:
            only_written(*outs[k])
        else:
            assert (outs[k][1] == CANARY).all()
    return v


@pytest.mark.parametrize("T,n_in,n_out", [(1, 64, 64), (1, 2048, 512), (2, 8, 1), (7, 72, 60), (64, 256, 128),
                                          (65, 512, 264), (300, 136, 1000), (999, 1024, 1407), (2050, 384, 256),
                                          (4500, 256, 384)])
def test_backward_sizes(moe, T, n_in, n_out):
    backward(moe, T, n_in, n_out)
    backward(moe, T, n_in, n_out, act="none")
    backward(moe, T, n_in, n_out, act="gelu", out="f32", dx_dtype="f32", dw_dtype="f32")


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_backward_activations_and_types(moe, act):
    for out in ("bf16", "f32"):
        for dx in ("bf16", "f32"):
            for dw in ("bf16", "f32"):
                backward(moe, 330, 192, 264, act=act, out=out, dx_dtype=dx, dw_dtype=dw)


@pytest.mark.parametrize("T,n_in,n_out", [(1, 1, 1), (5, 65, 33), (130, 999, 301), (517, 131, 515)])
def test_backward_odd_features(moe, T, n_in, n_out):
    for act in ("none", "silu"):
        backward(moe, T, n_in, n_out, act=act)
    backward(moe, T, n_in, n_out, out="f32", dx_dtype="f32", dw_dtype="f32")


def test_backward_strides(moe):
    for act in ("none", "silu"):
        backward(moe, 300, 256, 192, act=act, ldx=264, ldw=512, ldy=1024)
        backward(moe, 300, 256, 192, act=act, ldx=257, ldw=259, ldy=195)
        backward(moe, 300, 256, 192, act=act, out="f32", ldy=193, off=1)


@pytest.mark.parametrize("want", [("dx",), ("dW",), ("dbias",), ("dx", "dW"), ("dW", "dbias"), ("dx", "dbias")])
def test_backward_parts(moe, want):
    for act in ("none", "relu"):
        backward(moe, 140, 128, 96, act=act, want=want)


def test_backward_no_tokens_gives_zero_weight_gradients(moe):
    cfg = moe.make_linear_config(0, 64, 32, dw_dtype="f32")
    ws = moe.alloc_linear_workspace(cfg)
    dW, db = torch.full((32, 64), CANARY, device="cuda"), torch.full((32,), CANARY, device="cuda")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    moe.moe_linear_backward(cfg, e, None, None, torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"), e, dW, db, ws)
    assert (dW == 0).all() and (db == 0).all()


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu"])
def test_gradients_against_differences(moe, act):
    """The kernels' gradients against central differences of the loss sum(y * dy) in float64,
    within the gradients' own bounds summed along the direction."""
    g = torch.Generator(device="cuda").manual_seed(9)
    T, i, o = 37, 96, 56
    x, W = rows(g, T, i, torch.bfloat16), rows(g, o, i, torch.bfloat16, std=i ** -0.5)
    b = torch.randn(o, generator=g, device="cuda")
    dy = rows(g, T, o, torch.float32)
    cfg = moe.make_linear_config(T, i, o, act=act, out_dtype="f32", dx_dtype="f32", dw_dtype="f32")
    ws = moe.alloc_linear_workspace(cfg)
    y, pre = torch.empty((T, o), device="cuda"), torch.empty((T, o), device="cuda")
    moe.moe_linear_forward(cfg, x, W, b, None, pre, y, ws)
    got = {"dx": torch.empty((T, i), device="cuda"), "dW": torch.empty((o, i), device="cuda"),
           "dbias": torch.empty(o, device="cuda")}
    moe.moe_linear_backward(cfg, x, W, pre, dy, got["dx"], got["dW"], got["dbias"], ws)
    at = [t.double() for t in (x, W, b)]
    ref = B.linear_backward(x, W, at[0] @ at[1].t() + at[2], dy, act, torch.float32, torch.float32, torch.float32)

    def loss(x, W, b):
        return float((B.act(x @ W.t() + b, act) * dy.double()).sum())

    for n, k in enumerate(("dx", "dW", "dbias")):
        u = torch.randn(at[n].shape, generator=g, device="cuda").double()
        h = 1e-5
        hi, lo = list(at), list(at)
        hi[n], lo[n] = at[n] + h * u, at[n] - h * u
        slope = (loss(*hi) - loss(*lo)) / (2 * h)
        # the saved z is off by the forward's rounding; its effect on the slope is below one of
        # 2^-8 of the terms, which the bound counts once more
        bound = float((2 * ref[k][1] * u.abs()).sum()) + 1e-5 * abs(slope)
        assert abs(slope - float((got[k].double() * u).sum())) < bound


def test_other_stream_and_graph_replay(moe):
    """The calls run on the stream they are given, and a captured pair replays on new data."""
    cfg = moe.make_linear_config(200, 256, 128, act="silu")
    g = torch.Generator(device="cuda").manual_seed(2)
    x, W, dy = rows(g, 200, 256, torch.bfloat16), rows(g, 128, 256, torch.bfloat16, std=0.06), rows(g, 200, 128, torch.bfloat16)
    y, pre, dx = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((200, 128), (200, 128), (200, 256)))
    dW, db = torch.zeros((128, 256), dtype=torch.bfloat16, device="cuda"), torch.zeros(128, device="cuda")
    ws = moe.alloc_linear_workspace(cfg)

    def both(stream):
        moe.moe_linear_forward(cfg, x, W, None, None, pre, y, ws, stream)
        moe.moe_linear_backward(cfg, x, W, pre, dy, dx, dW, db, ws, stream)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    both(s)
    s.synchronize()
    plain = [t.clone() for t in (y, pre, dx, dW, db)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(None)
    for t in (y, pre, dx, dW, db):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(plain, (y, pre, dx, dW, db)):
        assert torch.equal(a, b)
    x.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    ref, _, bound, _ = B.linear(x, W, None, None, "silu", torch.bfloat16)
    within("y", y, ref, bound)
    assert moe.moe_read_status(ws) == 0
