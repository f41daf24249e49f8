"""Normalisation of rows and its gradients: within the oracle's rounding bounds on every kind, type, width,
stride and alignment, with nothing written outside the results."""
import math

import pytest
import torch

from oracle import step_oracle as S
from tests.conftest import ensure_built

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def moe():
    ensure_built()
    import routing_shared_expert_gb300 as moe
    return moe


class Rows:
    """A [rows][cols] matrix inside a larger buffer whose other values must stay."""

    def __init__(self, rows, cols, dtype, ld=0, off=0, values=None):
        ld = ld or cols
        self.buf = torch.full((off + rows * ld + 24,), 7.0, dtype=dtype, device="cuda")
        self.v = self.buf[off:off + rows * ld].view(rows, ld)[:, :cols]
        if values is not None:
            self.v.copy_(values)

    def untouched_around(self):
        mine = torch.zeros_like(self.buf, dtype=torch.bool)
        mine.as_strided(self.v.shape, self.v.stride(), self.v.storage_offset())[:] = True
        return bool((self.buf[~mine] == 7.0).all())


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, *shape, scale=1.0, shift=0.0):
    return torch.randn(shape, generator=g, device="cuda") * scale + shift


def near(got, want, name):
    value, bound = want
    err = (got.double() - value).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(err[bad].max()), float((err / bound.clamp(min=1e-300)).max()))


def check(moe, T, d, kind="layer", x="bf16", stream=None, y="bf16", w="f32", bias=True, save_sum=True, lds=(0, 0, 0, 0),
          off=0, eps=1e-5, seed=0, shift=0.3, alias=None, dsum=True):
    """The forward and the backward call of one layer; lds: row strides of x, residual, sum, y."""
    g = gen(1000 * T + d + seed)
    X = Rows(T, d, DT[x], lds[0], off, rand(g, T, d, shift=shift))
    R = Rows(T, d, DT[stream], lds[1], off, rand(g, T, d)) if stream else None
    Sm = Rows(T, d, DT[stream], lds[2], off) if stream and save_sum else None
    Y = Rows(T, d, DT[y], lds[3], off)
    if alias == "sum=residual":
        Sm = R
    if alias == "sum=x":
        Sm = X
    if alias == "y=x":
        Y = X
    weight = rand(g, d, scale=0.2, shift=1.0).to(DT[w]) if w else None
    b = rand(g, d, scale=0.2).to(DT[w]) if w and bias else None
    mean = torch.full((T,), 7.0, device="cuda") if kind == "layer" else None
    rstd = torch.full((T,), 7.0, device="cuda")
    x0, r0 = X.v.clone(), R.v.clone() if R else None
    moe.moe_layernorm_forward(X.v, R.v if R else None, weight, b, eps, Sm.v if Sm else None, Y.v, mean, rstd, kind=kind)
    want = S.layernorm(x0, r0, weight, b, eps, kind, DT[stream] if Sm else None, DT[y])
    near(Y.v, want["y"], "y")
    near(rstd, want["rstd"], "rstd")
    if mean is not None:
        near(mean, want["mean"], "mean")
    if Sm:
        near(Sm.v, want["sum"], "sum")
        assert Sm.untouched_around()
    assert Y.untouched_around() and X.untouched_around()

    H = Sm or Rows(T, d, DT[x], lds[0], off, x0)
    hx = H.v.clone()
    st = DT[stream or x]
    dy = Rows(T, d, DT[y], lds[3], off, rand(g, T, d))
    ds = Rows(T, d, st, lds[1], off, rand(g, T, d)) if dsum else None
    dx = Rows(T, d, st, lds[2], off)
    if alias == "dx=dsum":
        dx = ds
    if alias == "dx=dy":
        dx = dy
    if alias == "dx=h":
        dx = H
    dy0, ds0 = dy.v.clone(), ds.v.clone() if ds else None
    dw = torch.full((d,), 7.0, device="cuda")
    db = torch.full((d,), 7.0, device="cuda")
    ws = moe.alloc_layernorm_workspace(T, d)
    ws[256:] = 0xFF           # NaN where partial sums are not written
    moe.moe_layernorm_backward(H.v, weight, mean, rstd, dy.v, ds.v if ds else None, dx.v, dw, db, ws, kind=kind)
    want = S.layernorm_backward(hx, weight, mean, rstd, dy0, ds0, kind, st)
    near(dx.v, want["dx"], "dx")
    near(dw, want["dweight"], "dweight")
    near(db, want["dbias"], "dbias")
    assert dx.untouched_around() and moe.moe_read_status(ws) == 0


SIZES = [(1, 1), (1, 2), (2, 7), (3, 8), (5, 31), (9, 32), (1, 2048), (2, 129), (33, 64), (17, 255), (130, 256),
         (40, 257), (21, 1000), (700, 96), (65, 1023), (19, 1024), (11, 1025), (7, 2049), (37, 4095), (10, 4096), (13, 7168),
         (6, 8200), (5, 16384), (4, 16385), (3, 20003), (2, 65536), (1500, 40), (3000, 8), (613, 520),
         (2, 16384), (3, 8640), (1, 5760), (17, 3387), (16, 905), (5, 841), (37, 379), (2000, 227), (400, 13760), (1, 16383)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_sizes(moe, T, d, kind):
    check(moe, T, d, kind)
    check(moe, T, d, kind, x="f32", stream="bf16", y="f32", dsum=False)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("stream", ["bf16", "f32", None])
@pytest.mark.parametrize("y", ["bf16", "f32"])
@pytest.mark.parametrize("w", ["bf16", "f32", None])
def test_types(moe, x, stream, y, w):
    for T, d in ((37, 264), (37, 131), (9, 2560), (9, 2563)):
        check(moe, T, d, "layer", x, stream, y, w)
        check(moe, T, d, "rms", x, stream, y, w, bias=False, dsum=stream is not None)


@pytest.mark.parametrize("lds", [(272, 264, 512, 320), (257, 257, 257, 257), (259, 261, 263, 265), (264, 257, 0, 0),
                                 (0, 0, 0, 300), (300, 300, 300, 300)])
@pytest.mark.parametrize("off", [0, 1, 3, 8])
@pytest.mark.parametrize("d", [256, 250])
def test_strides_and_offsets(moe, lds, off, d):
    check(moe, 19, d, "layer", "bf16", "bf16", "bf16", lds=lds, off=off)
    check(moe, 19, d, "rms", "f32", "bf16", "f32", lds=lds, off=off)


@pytest.mark.parametrize("d", [1, 2, 3, 4, 5, 6])
@pytest.mark.parametrize("T", [2, 3, 5, 9, 40])
def test_rows_narrower_than_a_group(moe, T, d):
    for off in (0, 1, 5):
        for ld in (d, d + 1, 8):
            check(moe, T, d, "layer", "bf16", "bf16", "bf16", lds=(ld, ld, ld, ld), off=off)
            check(moe, T, d, "rms", "f32", "f32", "f32", lds=(ld, ld, ld, ld), off=off)
            check(moe, T, d, "rms", "f32", "bf16", "f32", lds=(ld, ld, ld, ld), off=off)


@pytest.mark.parametrize("T,d", [(2, 1), (3, 2), (4, 3), (7, 5), (9, 6), (3, 257), (2, 4095)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_what_lies_around_the_rows_does_not_count(moe, T, d, dtype):
    """The same results whether zeros or NaN lie before, behind and between the rows."""
    g = gen(T + d)
    x, dy, w = rand(g, T, d).to(dtype), rand(g, T, d).to(dtype), rand(g, d)
    for off in range(4):
        for ld in (d, d + 3):
            seen = []
            for fill in (0.0, math.nan):
                X, DY = (torch.full((off + T * ld + 24,), fill, dtype=dtype, device="cuda") for _ in range(2))
                X, DY = (b[off:off + T * ld].view(T, ld)[:, :d] for b in (X, DY))
                X.copy_(x)
                DY.copy_(dy)
                y, dx = Rows(T, d, dtype, ld, off).v, Rows(T, d, dtype, ld, off).v
                mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
                dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
                moe.moe_layernorm_forward(X, None, w, None, 1e-5, None, y, mean, rstd)
                moe.moe_layernorm_backward(X, w, mean, rstd, DY, None, dx, dw, db, moe.alloc_layernorm_workspace(T, d))
                seen.append([t.clone() for t in (y, mean, rstd, dx, dw, db)])
            for a, b in zip(*seen):
                assert torch.equal(a, b) and torch.isfinite(a).all()


def test_strided_long_rows(moe):
    check(moe, 23, 5000, "layer", "bf16", "f32", "bf16", lds=(5001, 5001, 5001, 5001), off=5)
    check(moe, 23, 5000, "layer", "bf16", "f32", "bf16", lds=(5008, 5016, 5024, 5032))


@pytest.mark.parametrize("alias", ["sum=residual", "sum=x", "y=x", "dx=dsum", "dx=dy", "dx=h"])
@pytest.mark.parametrize("T,d", [(19, 512), (19, 515), (640, 96), (5, 9000), (3, 17001)])
def test_in_place(moe, alias, T, d):
    check(moe, T, d, "layer", "f32", "f32", "f32", alias=alias, save_sum=alias != "y=x")
    check(moe, T, d, "rms", "bf16", "bf16", "bf16", alias=alias, save_sum=alias != "y=x")


@pytest.mark.parametrize("d", [16384, 16383, 13000, 12001])
def test_long_fp32_rows(moe, d):
    """Rows whose operands fill, or do not fit, a processor's shared memory."""
    for T in (3, 400):
        check(moe, T, d, "layer", "f32", "f32", "f32")
        check(moe, T, d, "rms", "f32", "f32", "bf16")


def test_tiny_values_without_eps(moe):
    """rstd of 1e18 and above: its square leaves fp32's range, the gradient's products with it do not."""
    g = gen(11)
    for kind in ("layer", "rms"):
        h, dy = rand(g, 7, 300) * 1e-20, rand(g, 7, 300) * 1e-8
        y, dx, rstd = torch.empty_like(h), torch.empty_like(h), torch.empty(7, device="cuda")
        mean = torch.empty(7, device="cuda") if kind == "layer" else None
        hd = h.double()
        mu = hd.mean(1, keepdim=True) if kind == "layer" else 0
        rstd.copy_(((hd - mu) ** 2).mean(1) ** -0.5)       # the forward pass would square 1e-20 in fp32
        if mean is not None:
            mean.copy_(hd.mean(1))
        moe.moe_layernorm_backward(h, None, mean, rstd, dy, None, dx, None, None, moe.alloc_layernorm_workspace(7, 300), kind=kind)
        want, bound = S.layernorm_backward(h, None, mean, rstd, dy, None, kind, torch.float32)["dx"]
        assert torch.isfinite(dx).all()
        near(dx, (want, bound), kind)


def test_a_sum_that_is_not_stored(moe):
    check(moe, 31, 777, "layer", "bf16", "bf16", "f32", save_sum=False)
    check(moe, 31, 768, "rms", "f32", "bf16", "bf16", save_sum=False)


def test_a_mean_far_from_the_spread(moe):
    """A mean of 4096 with a spread of 1 in fp32: E h^2 - mean^2 in fp32 would leave nothing of the variance."""
    check(moe, 40, 1000, "layer", "f32", None, "f32", shift=4096.0)
    check(moe, 40, 4096, "layer", "f32", None, "f32", shift=4096.0)


def test_constant_and_zero_rows(moe):
    for v in (0.0, 3.0):
        x = torch.full((3, 300), v, device="cuda")
        y = torch.empty_like(x)
        mean, rstd = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
        moe.moe_layernorm_forward(x, None, None, None, 1e-5, None, y, mean, rstd)
        assert torch.equal(mean, torch.full_like(mean, v)) and torch.equal(y, torch.zeros_like(y))
        assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=4 * 2.0 ** -24)
    moe.moe_layernorm_forward(torch.zeros_like(x), None, None, None, 0.0, None, y, None, rstd, kind="rms")
    assert torch.isinf(rstd).all() and torch.isnan(y).all()      # 0 / 0, as the formula has it


@pytest.mark.parametrize("d", [64, 100, 2048, 5001, 17000])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_broken_rows_stay_alone(moe, d, bad):
    g = gen(d)
    x = rand(g, 20, d)
    x[3, d // 2] = bad
    x[11, 0] = bad
    x[12, d - 1] = bad
    y, mean, rstd = torch.empty_like(x), torch.empty(20, device="cuda"), torch.empty(20, device="cuda")
    moe.moe_layernorm_forward(x, None, None, None, 1e-5, None, y, mean, rstd)
    broken = torch.zeros(20, dtype=torch.bool, device="cuda")
    broken[[3, 11, 12]] = True
    assert torch.isnan(y[broken]).all() and torch.isfinite(y[~broken]).all()
    moe.moe_layernorm_forward(x, None, None, None, 1e-5, None, y, None, rstd, kind="rms")
    assert torch.isnan(y[3, d // 2]) and torch.isfinite(y[~broken]).all()
    dy = rand(g, 20, d)
    moe.moe_layernorm_forward(torch.nan_to_num(x, 0, 0, 0), None, None, None, 1e-5, None, y, mean, rstd)
    dy[5, 1] = bad
    dx, dw, db = torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = moe.alloc_layernorm_workspace(20, d)
    moe.moe_layernorm_backward(torch.nan_to_num(x, 0, 0, 0), None, mean, rstd, dy, None, dx, dw, db, ws)
    # infinite sums: every value of the row is an infinity or a NaN
    assert not torch.isfinite(dx[5]).any() and torch.isfinite(dx[[4, 6]]).all()
    assert not torch.isfinite(dw[1]) and not torch.isfinite(db[1]) and torch.isfinite(db[2:]).all()


@pytest.mark.parametrize("T,d", [(33, 200), (5, 2049), (300, 64)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradient_against_differences(moe, T, d, kind):
    """The forward kernel's difference quotient against the backward kernel's gradient: apart by the roundings of
    y over the step, and by the quotient's own distance from the derivative, which the oracle gives."""
    g = gen(5)
    h, u, dy = rand(g, T, d), rand(g, T, d), rand(g, T, d)
    w, b = rand(g, d, scale=0.2, shift=1.0), rand(g, d, scale=0.2)
    s = 2.0 ** -7
    ys, wants = [], []
    for sign in (1, -1):
        x = h + sign * s * u
        y = torch.empty_like(x)
        moe.moe_layernorm_forward(x, None, w, b, 1e-5, None, y, None, None, kind=kind)
        ys.append((x, y))
        wants.append(S.layernorm(x, None, w, b, 1e-5, kind, None, torch.float32)["y"])
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    y, dx = torch.empty_like(h), torch.empty_like(h)
    moe.moe_layernorm_forward(h, None, w, b, 1e-5, None, y, mean if kind == "layer" else None, rstd, kind=kind)
    moe.moe_layernorm_backward(h, w, mean, rstd, dy, None, dx, None, None, moe.alloc_layernorm_workspace(T, d), kind=kind)
    step = (ys[0][0].double() - ys[1][0].double()) / 2          # s u as the inputs hold it
    slope = float(((ys[0][1].double() - ys[1][1].double()) / 2 * dy.double()).sum())
    exact_slope = float(((wants[0][0] - wants[1][0]) / 2 * dy.double()).sum())
    want_dx, e_dx = S.layernorm_backward(h, w, mean, rstd, dy, None, kind, torch.float32)["dx"]
    # the statistics that the oracle's gradient is given are the kernel's: off by their own bound
    e = S.layernorm(h, None, w, b, 1e-5, kind, None, torch.float32)["rstd"]
    e_rel = 8 * float((e[1] / e[0]).max())
    bound = float(((wants[0][1] + wants[1][1]) / 2 * dy.double().abs()).sum())
    bound += float(((e_dx + e_rel * (want_dx.abs() + (rstd[:, None] * dy * w).abs())) * step.abs()).sum())
    bound += abs(exact_slope - float((want_dx * step).sum()))
    assert abs(slope - float((dx.double() * step).sum())) <= bound
    assert bound < 0.05 * abs(float((dy.double() * step).norm())) + 1.0     # the bound says something


@pytest.mark.parametrize("T,d", [(33, 200), (5, 2049), (300, 64), (3, 17000)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradients_against_differences_along_themselves(moe, T, d, kind):
    """The forward kernel's difference quotients along the gradients: the slope is as large as it can be there, and what
    is allowed between the two kernels, the roundings of y over the step and of the gradient, is under a fiftieth of it (at
    most 0.011, from the oracles alone).

    With rows of spread near 1 and steps of s = 2^-7 in units of it, a central difference is off by s^2 / 6 of the third
    derivative, which is of the size of 15 |dy| per unit step: under 3e-4 of the slope, where |dx| is half of |dy| or more."""
    g = gen(15)
    h, dy = rand(g, T, d), rand(g, T, d)
    w, b = rand(g, d, scale=0.2, shift=1.0), rand(g, d, scale=0.2)
    mean = torch.empty(T, device="cuda") if kind == "layer" else None
    y, rstd, dx = torch.empty_like(h), torch.empty(T, device="cuda"), torch.empty_like(h)
    dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    moe.moe_layernorm_forward(h, None, w, b, 1e-5, None, y, mean, rstd, kind=kind)
    moe.moe_layernorm_backward(h, w, mean, rstd, dy, None, dx, dw, db, moe.alloc_layernorm_workspace(T, d), kind=kind)
    exact = S.layernorm(h, None, w, b, 1e-5, kind, None, torch.float32)
    true_mean = exact["mean"][0] if kind == "layer" else None
    want = S.layernorm_backward(h, w, true_mean, exact["rstd"][0], dy, None, kind, torch.float32)
    # the kernel's statistics are off by their own bounds, and its gradients by what that makes
    e_rel = 8 * float((exact["rstd"][1] / exact["rstd"][0]).max())
    grown = {"dx": e_rel * (want["dx"][0].abs() + (rstd[:, None] * dy * w).abs().double()), "dbias": 0.0,
             "dweight": e_rel * (dy.double().abs() * (1 + y.double().abs() + h.double().abs())).sum(0)}
    for name, got in (("dx", dx), ("dweight", dw), ("dbias", db)):
        G, e = want[name]
        u = (G / G.square().mean().sqrt() * 2.0 ** -7).float()
        sides = []
        for sign in (1, -1):
            x, w2, b2 = (t + sign * u if name == n else t for n, t in (("dx", h), ("dweight", w), ("dbias", b)))
            moved = {"dx": x, "dweight": w2, "dbias": b2}[name]
            out = torch.empty_like(y)
            moe.moe_layernorm_forward(x, None, w2, b2, 1e-5, None, out, None, None, kind=kind)
            sides.append((moved.double(), out.double(), *S.layernorm(x, None, w2, b2, 1e-5, kind, None, torch.float32)["y"]))
        step = (sides[0][0] - sides[1][0]) / 2          # as the inputs hold it
        slope = float(((sides[0][1] - sides[1][1]) / 2 * dy.double()).sum())
        exact_slope = float(((sides[0][2] - sides[1][2]) / 2 * dy.double()).sum())
        along = float((got.double() * step).sum())
        # the oracles' own derivative and quotient
        assert abs(float((G * step).sum()) - exact_slope) <= 1e-3 * exact_slope, name
        bound = float(((sides[0][3] + sides[1][3]) / 2 * dy.double().abs()).sum()) + float(((e + grown[name]) * step.abs()).sum())
        assert bound <= 0.02 * exact_slope, (name, bound, exact_slope)
        assert abs(slope - along) <= bound + 1e-3 * exact_slope, (name, slope, along, bound)


def test_parts_that_are_not_asked_for(moe):
    """Every subset of the results gives the values of the full call."""
    g = gen(6)
    for T, d in ((50, 128), (50, 129), (3, 18000)):
        h, dy, w = rand(g, T, d), rand(g, T, d), rand(g, d)
        y, mean, rstd = torch.empty_like(h), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        moe.moe_layernorm_forward(h, None, w, None, 1e-5, None, y, mean, rstd)
        y2 = torch.empty_like(y)
        moe.moe_layernorm_forward(h, None, w, None, 1e-5, None, y2, None, None)
        assert torch.equal(y, y2)
        ws = moe.alloc_layernorm_workspace(T, d)
        full = [torch.empty_like(h), torch.empty_like(w), torch.empty_like(w)]
        moe.moe_layernorm_backward(h, w, mean, rstd, dy, None, *full, ws)
        for mask in range(8):
            part = [torch.full_like(t, 7.0) if mask >> i & 1 else None for i, t in enumerate(full)]
            moe.moe_layernorm_backward(h, w, mean, rstd, dy, None, *part, ws)
            for p, f in zip(part, full):
                assert p is None or torch.equal(p, f)


def test_calls_repeat_bit_for_bit_and_in_a_graph_on_another_stream(moe):
    g = gen(7)
    T, d = 2000, 768
    h, dy, w = rand(g, T, d).bfloat16(), rand(g, T, d).bfloat16(), rand(g, d)
    y, rstd, dx = torch.empty_like(h), torch.empty(T, device="cuda"), torch.empty_like(h)
    dw, ws = torch.empty(d, device="cuda"), moe.alloc_layernorm_workspace(T, d)

    def step():
        moe.moe_layernorm_forward(h, None, w, None, 1e-6, None, y, None, rstd, kind="rms")
        moe.moe_layernorm_backward(h, w, None, rstd, dy, None, dx, dw, None, ws, kind="rms")

    step()
    first = [t.clone() for t in (y, rstd, dx, dw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for t in (y, rstd, dx, dw):
            t.zero_()
        graph.replay()
    torch.cuda.current_stream().wait_stream(side)
    for t, f in zip((y, rstd, dx, dw), first):
        assert torch.equal(t, f)
    h.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(dx, first[2])       # new inputs are read


def test_graphs_of_few_rows_share_a_workspace(moe):
    """Calls of several shapes, captured with one workspace and replayed in turn, leave it ready for one another."""
    g = gen(9)
    ws = moe.alloc_layernorm_workspace(300, 512)
    calls = []
    for T, d in ((5, 512), (31, 500), (1, 64), (300, 96), (260, 512)):
        h, dy = rand(g, T, d), rand(g, T, d)
        rstd, dw, db = torch.rand(T, device="cuda", generator=g) + 0.5, torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        mean = torch.zeros(T, device="cuda")
        args = (h, None, mean, rstd, dy, None, None, dw, db, ws)
        moe.moe_layernorm_backward(*args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_layernorm_backward(*args)
        calls.append((graph, args))
    for _ in range(2):
        for graph, (h, _, mean, rstd, dy, _, _, dw, db, _) in calls + calls[::-1]:
            dw.fill_(7.0)
            db.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            want = S.layernorm_backward(h, None, mean, rstd, dy, None, "layer", torch.float32)
            near(dw, want["dweight"], "dw")
            near(db, want["dbias"], "db")
    assert moe.moe_read_status(ws) == 0


@pytest.mark.parametrize("x,stream,y", [("bf16", None, "bf16"), ("bf16", "bf16", "bf16"), ("f32", "bf16", "bf16"), ("f32", "f32", "f32")])
@pytest.mark.parametrize("d", [8, 256, 520, 1024, 4096, 7168])
def test_a_row_has_the_same_bits_in_every_call(moe, x, stream, y, d):
    """Rows on groups of eight: a token's results do not depend on how many rows are normalised with it, nor on its place
    among them."""
    g = gen(d)
    T = 6000
    X, R = rand(g, T, d, shift=0.3).to(DT[x]), rand(g, T, d).to(DT[stream]) if stream else None
    w, b = rand(g, d, scale=0.2, shift=1.0), rand(g, d, scale=0.2)

    def call(rows, kind, bias):
        x, r = X[rows], R[rows] if stream else None
        out = dict(y=torch.empty_like(x, dtype=DT[y]), rstd=torch.empty(len(x), device="cuda"))
        mean = out["mean"] = torch.zeros(len(x), device="cuda")
        out["sum"] = torch.empty_like(r) if stream else mean
        moe.moe_layernorm_forward(x, r, w, bias, 1e-5, out["sum"] if stream else None, out["y"],
                                  mean if kind == "layer" else None, out["rstd"], kind=kind)
        return out

    order = torch.randperm(T, generator=g, device="cuda")
    for kind in ("layer", "rms"):
        for bias in (b, None):
            whole = call(torch.arange(T, device="cuda"), kind, bias)
            for part in (order, order[:1], order[:3], order[5:170], order[:1300]):
                for name, got in call(part, kind, bias).items():
                    assert torch.equal(got, whole[name][part]), (kind, bias is None, len(part), name)


def test_no_rows(moe):
    x, v = torch.empty((0, 8), device="cuda"), torch.empty(0, device="cuda")
    dw, db = torch.ones(8, device="cuda"), torch.ones(8, device="cuda")
    moe.moe_layernorm_forward(x, None, None, None, 1e-5, None, x, v, v)
    moe.moe_layernorm_backward(x, None, v, v, x, None, x, dw, db, moe.alloc_layernorm_workspace(0, 8))
    assert not dw.any() and not db.any()


def test_offsets_past_32_bits(moe):
    """Rows whose elements lie past 2^31: the last rows are those of a call on them alone."""
    T, d = 70000, 32768
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    g = gen(8)
    for a in range(0, T, 10000):
        x[a:a + 10000] = torch.randn((10000, d), generator=g, device="cuda").bfloat16()
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    moe.moe_layernorm_forward(x, None, None, None, 1e-6, None, y, None, rstd, kind="rms")
    y2, r2 = torch.empty_like(x[:9]), torch.empty(9, device="cuda")
    moe.moe_layernorm_forward(x[-9:], None, None, None, 1e-6, None, y2, None, r2, kind="rms")
    assert torch.equal(y[-9:], y2) and torch.equal(rstd[-9:], r2)
    near(y2, S.layernorm(x[-9:], None, None, None, 1e-6, "rms", None, torch.bfloat16)["y"], "y")
    dx = torch.empty_like(x)
    moe.moe_layernorm_backward(x, None, None, rstd, y, None, dx, None, None, moe.alloc_layernorm_workspace(T, d), kind="rms")
    near(dx[-9:], S.layernorm_backward(x[-9:], None, None, r2, y2, None, "rms", torch.bfloat16)["dx"], "dx")
