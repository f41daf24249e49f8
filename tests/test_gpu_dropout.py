"""Dropout from the counter-based generator: the mask is the published generator's bit for bit,
the values are within the oracle's rounding bounds, on every type, stride and tail."""
import math

import pytest
import torch

from oracle import block_oracle as B
from tests.conftest import ensure_built

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SEED, OFFSET = 0x1234567890ABCDEF, 0x7EDCBA9876543210


@pytest.fixture(scope="module")
def moe():
    ensure_built()
    import routing_shared_expert_gb300 as moe
    return moe


def state(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def strided(shape, dtype, ld=None, off=0, fill=None, g=None):
    rows, cols = shape
    ld = ld or cols
    buf = torch.full((off + rows * ld + 16,), 7.0, dtype=dtype, device="cuda")
    v = buf[off:off + rows * ld].view(rows, ld)[:, :cols]
    if g is not None:
        v.copy_(torch.randn(shape, generator=g, device="cuda"))
    return v, buf


def check(moe, rows, cols, p, x="f32", r="bf16", y="bf16", ldx=None, ldr=None, ldy=None, off=0, in_place=None):
    g = torch.Generator(device="cuda").manual_seed(rows * 31 + cols)
    xs, _ = strided((rows, cols), DT[x], ldx, off, g=g)
    rs, _ = strided((rows, cols), DT[r], ldr, off, g=g) if r else (None, None)
    ys, buf = strided((rows, cols), DT[y], ldy, off)
    x0, r0 = xs.clone(), rs.clone() if r else None
    if in_place == "x":
        ys = xs
    if in_place == "r":
        ys = rs
    moe.moe_dropout_add(xs, rs, p, state(), ys)
    ref, bound = B.dropout(x0, r0, p, SEED, OFFSET, DT[y])
    err = (ys.double() - ref).abs()
    assert (err <= bound).all(), float((err - bound).max())
    if in_place is None:
        keep = torch.zeros_like(buf, dtype=torch.bool)
        keep.as_strided(ys.shape, ys.stride(), ys.storage_offset())[:] = True
        assert (buf[~keep] == 7.0).all()
    # the backward pass takes the same mask
    dy, _ = strided((rows, cols), DT[y], ldy, off, g=g)
    dx, dbuf = strided((rows, cols), DT[x], ldx, off)
    moe.moe_dropout_backward(dy, p, state(), dx)
    ref, bound = B.dropout(dy, None, p, SEED, OFFSET, DT[x])
    assert ((dx.double() - ref).abs() <= bound).all()
    keep = torch.zeros_like(dbuf, dtype=torch.bool)
    keep.as_strided(dx.shape, dx.stride(), dx.storage_offset())[:] = True
    assert (dbuf[~keep] == 7.0).all()


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 3), (1, 4), (1, 5), (2, 7), (3, 8), (5, 64), (7, 33), (64, 100),
                                       (129, 1023), (1000, 256), (77, 4099),
                                       (1025, 2049), (300, 8192)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_sizes(moe, rows, cols, p):
    check(moe, rows, cols, p)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("r", ["f32", "bf16", None])
@pytest.mark.parametrize("y", ["f32", "bf16"])
def test_types(moe, x, r, y):
    check(moe, 37, 264, 0.25, x, r, y)
    check(moe, 37, 131, 0.25, x, r, y)


@pytest.mark.parametrize("kw", [dict(ldx=272, ldr=264, ldy=512), dict(ldx=257, ldr=259, ldy=261), dict(off=1),
                                dict(off=8, ldx=264), dict(ldy=300), dict(off=3, ldr=333), dict(ldx=258, ldr=258, ldy=258)])
@pytest.mark.parametrize("cols", [256, 250])
def test_strides_and_offsets(moe, kw, cols):
    for y in ("bf16", "f32"):
        check(moe, 19, cols, 0.3, y=y, **kw)


def test_in_place(moe):
    check(moe, 21, 200, 0.2, x="bf16", r="bf16", y="bf16", in_place="x")
    check(moe, 21, 203, 0.2, x="f32", r="f32", y="f32", in_place="r")


def test_dropped_values_are_not_looked_at(moe):
    x = torch.full((8, 128), float("nan"), device="cuda")
    keep = B.keep_mask(8, 128, 0.5, SEED, OFFSET).cuda()
    x[keep] = 1.0
    y = torch.empty_like(x)
    moe.moe_dropout_add(x, None, 0.5, state(), y)
    assert torch.equal(y, keep.float() * 2)
    x[~keep] = float("inf")
    moe.moe_dropout_add(x, None, 0.5, state(), y)
    assert torch.equal(y, keep.float() * 2)


def test_threshold_is_exact(moe):
    """At p = word / 2^32 the element is kept, at (word + 1) / 2^32 it is dropped."""
    x, y = torch.ones((1, 4), device="cuda"), torch.empty((1, 4), device="cuda")
    words = B.philox([0], SEED, OFFSET)[0]
    for j in range(4):
        for step, kept in ((0, True), (1, False)):
            moe.moe_dropout_add(x, None, (int(words[j]) + step) / 2.0 ** 32, state(), y)
            assert bool(y[0, j] != 0) == kept


def test_seed_and_offset_change_the_mask_and_a_graph_reads_them_anew(moe):
    x = torch.ones((64, 64), device="cuda")
    rng, y = state(1, 0), torch.empty_like(x)
    moe.moe_dropout_add(x, None, 0.5, rng, y)
    first = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_dropout_add(x, None, 0.5, rng, y)
    graph.replay()
    assert torch.equal(y, first)
    for seed, offset in ((2, 0), (1, 1), (1, 1 << 40), (1 << 40, 0), (-1, -1)):
        rng.copy_(torch.tensor([seed, offset], dtype=torch.int64))
        graph.replay()
        want = B.keep_mask(64, 64, 0.5, seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)).cuda()
        assert torch.equal(y != 0, want)


def test_gradient_against_differences(moe):
    """y is linear in x: the gradient equals the difference quotient up to fp32 rounding."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, u, dy = (torch.randn((33, 70), generator=g, device="cuda") for _ in range(3))
    hi, lo, dx = (torch.empty_like(x) for _ in range(3))
    moe.moe_dropout_add(x + u, None, 0.4, state(), hi)
    moe.moe_dropout_add(x - u, None, 0.4, state(), lo)
    moe.moe_dropout_backward(dy, 0.4, state(), dx)
    slope = float(((hi.double() - lo.double()) / 2 * dy.double()).sum())
    # each of hi, lo carries the roundings of x +- u, the scale and the product
    bound = float((4 * B.EPS32 * (hi.double().abs() + lo.double().abs()) * dy.double().abs()).sum())
    bound += float((2 * B.EPS32 * (dx.double() * u.double()).abs()).sum())
    assert abs(slope - float((dx.double() * u.double()).sum())) <= bound


def test_elements_past_32_bits_of_bytes(moe):
    """Over 2^31 elements: the element number and the offsets need 64 bits."""
    rows, cols = 66000, 32768
    assert rows * cols > 2 ** 31
    x = torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(x)
    moe.moe_dropout_add(x, None, 0.5, state(), y)
    for r0 in (0, 33000, rows - 2):
        first = r0 * cols // 4
        words = B.philox(range(first, first + 2 * cols // 4), SEED, OFFSET).reshape(2, cols)
        want = torch.from_numpy(words >= 2 ** 31).cuda()
        assert torch.equal(y[r0:r0 + 2] != 0, want)
    assert math.isclose(float(y[::97].float().mean()), 1.0, abs_tol=0.01)


def test_wrapper_refusals(moe):
    x = torch.zeros((4, 6), device="cuda")
    with pytest.raises(ValueError):
        moe.moe_dropout_add(x, None, 0.1, state(), torch.zeros((4, 7), device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_dropout_add(x.t(), None, 0.1, state(), torch.zeros((6, 4), device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_dropout_add(x.half(), None, 0.1, state(), x)
    with pytest.raises(ValueError):
        moe.moe_dropout_add(x, None, 0.1, torch.zeros(2, device="cuda"), x)
    with pytest.raises(moe.MoEError):
        moe.moe_dropout_add(x, None, 1.1, state(), x)
