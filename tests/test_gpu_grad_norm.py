"""The global gradient norm and clipping: within the oracle's rounding bounds over lists of every kind."""
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


def check(moe, grads, max_norm, in_place, ws=None):
    """grads: list of Rows."""
    views = [g.v for g in grads]
    before = [v.clone() for v in views]
    norm = torch.full((2,), 7.0, device="cuda")
    ws = moe.alloc_grad_norm_workspace() if ws is None else ws
    want, coef, rel_n, rel_c = S.grad_norm(before, max_norm)
    outs = grads if in_place else [Rows(*v.shape, v.dtype, v.shape[1] + 3 * (i % 2), i % 4) for i, v in enumerate(views)]
    moe.moe_grad_norm(views, norm, ws, max_norm)
    alone = norm.clone()
    moe.moe_clip_grad_norm(views, max_norm, None if in_place else [o.v for o in outs], norm, ws)
    assert torch.equal(alone, norm)
    assert abs(float(norm[0]) - want) <= rel_n * want, (float(norm[0]), want)
    assert abs(float(norm[1]) - coef) <= rel_c * coef
    for o, w in zip(outs, S.clip(before, max_norm)):
        near(o.v, w, "out")
        assert o.untouched_around()
    if not in_place or float(norm[1]) == 1.0:
        for v, b in zip(views, before):
            assert torch.equal(v, b)
    assert moe.moe_read_status(ws) == 0


SHAPES = [[(1, 1)], [(1, 7)], [(3, 5), (1, 1)], [(1, 8191), (1, 8192), (1, 8193)], [(300, 129), (2, 2), (1, 100000)],
          [(64, 64)] * 7, [(1, 3)] * 56, [(1, 3)] * 57, [(2, 5)] * 200 + [(700, 1000)], [(1, 33)] * 1300, [(1000, 4096)] * 5]


@pytest.mark.parametrize("shapes", SHAPES, ids=[f"{len(s)}x{s[0][0]}x{s[0][1]}" for s in SHAPES])
@pytest.mark.parametrize("in_place", [False, True])
def test_lists(moe, shapes, in_place):
    g = gen(len(shapes))
    for max_norm in (1.0, 1e9):
        for types in (("f32",), ("bf16",), ("bf16", "f32")):
            grads = [Rows(r, c, DT[types[i % len(types)]], values=rand(g, r, c, scale=0.1 + i % 3))
                     for i, (r, c) in enumerate(shapes)]
            check(moe, grads, max_norm, in_place)


@pytest.mark.parametrize("off", [0, 1, 2, 3, 5, 8])
@pytest.mark.parametrize("in_place", [False, True])
def test_alignment_and_strides(moe, off, in_place):
    g = gen(off)
    for t in ("f32", "bf16"):
        grads = [Rows(r, c, DT[t], ld, off, rand(g, r, c))
                 for r, c, ld in ((1, 20000, 0), (40, 64, 72), (40, 64, 65), (3, 9001, 9001), (9000, 3, 4), (500, 1, 2))]
        check(moe, grads, 0.5, in_place)


def test_columns_of_one_matrix(moe):
    """Views of neighbouring columns share no memory and are both clipped."""
    both = rand(gen(1), 100, 256)
    before = both.clone()
    norm, ws = torch.empty(2, device="cuda"), moe.alloc_grad_norm_workspace()
    moe.moe_clip_grad_norm([both[:, :100], both[:, 100:]], 1.0, None, norm, ws)
    near(both, S.clip([before], 1.0)[0], "both")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tensors_in_the_gaps_of_another(moe, dtype):
    """A matrix, and between its rows a single row and a matrix of another stride."""
    both = rand(gen(3), 100, 256).to(dtype)
    before = both.clone()
    parts = lambda t: [t[:, :100], t[0:1, 100:], t[1::2, 101:200]]
    norm, ws = torch.empty(2, device="cuda"), moe.alloc_grad_norm_workspace()
    moe.moe_clip_grad_norm(parts(both), 1.0, None, norm, ws)
    mine = torch.zeros_like(before, dtype=torch.bool)
    for p, m, w in zip(parts(both), parts(mine), S.clip(parts(before), 1.0)):
        near(p, w, "part")
        m[:] = True
    assert torch.equal(both[~mine], before[~mine])


def test_shapes_of_any_rank_and_empty_tensors(moe):
    g = gen(2)
    ws = moe.alloc_grad_norm_workspace()
    grads = [rand(g, 4, 5, 6), rand(g, 10), torch.empty((0, 4), device="cuda"), rand(g, 1, 1)[0, 0], torch.empty(0, device="cuda")]
    out = [torch.full_like(t, 7.0) for t in grads]
    norm = torch.empty(2, device="cuda")
    moe.moe_clip_grad_norm(grads, 1.0, out, norm, ws)
    for o, w in zip(out, S.clip(grads, 1.0)):
        near(o, w, "out")
    for none in ([], [torch.empty(0, device="cuda")]):
        moe.moe_clip_grad_norm(none, 1.0, None, norm, ws)
        assert norm.tolist() == [0.0, 1.0]


def test_the_factor(moe):
    ws, norm = moe.alloc_grad_norm_workspace(), torch.empty(2, device="cuda")
    g = torch.full((16,), 2.0, device="cuda")           # norm 8
    for most, coef in ((math.inf, 1.0), (8.0, 8.0 / 8.000001), (4.0, 4.0 / 8.000001), (16.0, 1.0), (0.0, 0.0)):
        moe.moe_grad_norm([g], norm, ws, most)
        assert float(norm[0]) == 8.0 and abs(float(norm[1]) - coef) <= 2.0 ** -23 * coef
    moe.moe_clip_grad_norm([g], 0.0, None, norm, ws)
    assert not g.any()
    moe.moe_clip_grad_norm([g], 1.0, None, norm, ws)
    assert norm.tolist() == [0.0, 1.0]
    z = torch.zeros(5, device="cuda")
    moe.moe_clip_grad_norm([z], 0.0, None, norm, ws)     # 0 / 1e-6
    assert norm.tolist() == [0.0, 0.0]


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", [0, 4097, 9999])
def test_broken_gradients_show(moe, bad, where):
    g = rand(gen(3), 10000)
    g[where] = bad
    other = torch.ones((5, 5), dtype=torch.bfloat16, device="cuda")
    out = [torch.empty_like(g), torch.empty_like(other)]
    norm, ws = torch.empty(2, device="cuda"), moe.alloc_grad_norm_workspace()
    moe.moe_clip_grad_norm([g, other], 1.0, out, norm, ws)
    if math.isnan(bad):
        assert torch.isnan(norm).all() and torch.isnan(out[1]).all() and torch.isnan(out[0]).all()
    else:       # the factor is 0: finite gradients vanish, 0 times infinity does not
        assert float(norm[0]) == math.inf and float(norm[1]) == 0.0
        assert not out[1].any() and torch.isnan(out[0][where]) and int(torch.isnan(out[0]).sum()) == 1


def test_large_and_small_squares(moe):
    """Squares past fp32's range: an infinite norm, as the header says; the largest that stay inside are right."""
    norm, ws = torch.empty(2, device="cuda"), moe.alloc_grad_norm_workspace()
    moe.moe_grad_norm([torch.full((3,), 1e20, device="cuda")], norm, ws, 1.0)
    assert norm.tolist() == [math.inf, 0.0]
    g = torch.full((100000,), 1e17, device="cuda")      # squares sum to 1e39 over the tensor, past fp32
    moe.moe_grad_norm([g], norm, ws, 1.0)
    assert abs(float(norm[0]) / (1e17 * math.sqrt(1e5)) - 1) < 1e-5
    moe.moe_grad_norm([torch.full((100,), 1e-15, device="cuda")], norm, ws, 1.0)
    assert abs(float(norm[0]) / 1e-14 - 1) < 1e-5 and float(norm[1]) == 1.0


def test_calls_repeat_bit_for_bit_and_in_graphs_that_share_a_workspace(moe):
    g = gen(4)
    a = [rand(g, 3000, 700), rand(g, 999), rand(g, 50, 50).bfloat16()]
    b = [rand(g, 20), rand(g, 777, 77).bfloat16()]
    ws = moe.alloc_grad_norm_workspace()
    na, nb = torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
    oa, ob = [torch.empty_like(t) for t in a], [torch.empty_like(t) for t in b]
    graphs = []
    for grads, out, norm in ((a, oa, na), (b, ob, nb)):
        moe.moe_clip_grad_norm(grads, 1.0, out, norm, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_clip_grad_norm(grads, 1.0, out, norm, ws)
        graphs.append(graph)
    torch.cuda.synchronize()
    first = [t.clone() for t in (na, nb, *oa, *ob)]
    for _ in range(3):
        for t in (na, nb, *oa, *ob):
            t.fill_(7.0)
        for graph in graphs + graphs[::-1]:
            graph.replay()
        torch.cuda.synchronize()
        for t, f in zip((na, nb, *oa, *ob), first):
            assert torch.equal(t, f)
    a[0].mul_(3)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert abs(float(na[0]) - S.grad_norm(a, 1.0)[0]) < 1e-3 * float(na[0])


def test_a_captured_clip_in_place_leaves_clipped_gradients_alone(moe):
    """Replayed, the second pass has nothing to scale; new gradients are scaled again."""
    v = rand(gen(5), 5000)
    norm, ws = torch.empty(2, device="cuda"), moe.alloc_grad_norm_workspace()
    graph = torch.cuda.CUDAGraph()
    keep = v.clone()
    with torch.cuda.graph(graph):
        moe.moe_clip_grad_norm([v], 1.0, None, norm, ws)
    graph.replay()
    torch.cuda.synchronize()
    near(v, S.clip([keep], 1.0)[0], "first")
    v.copy_(keep * 1e-4)
    want = v.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert float(norm[1]) == 1.0 and torch.equal(v, want)


def test_more_than_32_bits_of_elements(moe):
    n = 2 ** 31 + 4099
    g = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    tail = torch.full((3,), 2.0, device="cuda")
    norm, ws = torch.empty(2, device="cuda"), moe.alloc_grad_norm_workspace()
    moe.moe_clip_grad_norm([g, tail], 1.0, None, norm, ws)
    want = math.sqrt(n + 12)
    # every thread's squares are ones: whole numbers below 2^24 are exact in fp32
    assert abs(float(norm[0]) / want - 1) < 2 * 2.0 ** -24
    v = float((torch.ones(1) / want).bfloat16())
    assert abs(float(g[0]) / v - 1) < 2.0 ** -7
    for a in range(0, n, 1 << 28):
        assert (g[a:a + (1 << 28)] == g[0]).all()
