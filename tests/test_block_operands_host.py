"""What the wrappers of the block operators refuse before the library sees it (no GPU): operands
whose memory does not hold what the call would read or write.  Host tensors that say they are
on the GPU stand for device tensors; a refused call never looks at what their addresses hold."""
import pytest
import torch

from tests.conftest import ensure_built


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)


def dev(t):
    return t.as_subclass(OnDevice)


@pytest.fixture(scope="module")
def nat():
    ensure_built()
    from routing_shared_expert_gb300 import _native
    return _native


RNG = torch.zeros(2, dtype=torch.int64)


def overlapping(kind, rows, cols):
    """A [rows][cols] matrix whose rows share memory."""
    if kind == "expanded":
        return torch.zeros(cols).expand(rows, cols)
    if kind == "one value":
        return torch.zeros(1, 1).expand(rows, cols)
    return torch.zeros(rows + cols).as_strided((rows, cols), (1, 1))


@pytest.mark.parametrize("kind", ["expanded", "one value", "window"])
@pytest.mark.parametrize("cols", [1, 64])
@pytest.mark.parametrize("which", ["x", "residual", "y", "dy", "dx"])
def test_dropout_refuses_rows_that_overlap(nat, which, cols, kind):
    """A row stride below the row's length: 0 would mean dense rows to the library, which would
    then walk rows * cols elements of a buffer of cols."""
    if kind == "window" and cols == 1:
        return                        # dense: a stride of one element
    rows = 1000
    o = {k: dev(torch.zeros(rows, cols)) for k in ("x", "residual", "y", "dy", "dx")}
    o[which] = dev(overlapping(kind, rows, cols))
    if which in ("x", "residual", "y"):
        with pytest.raises(ValueError, match="rows"):
            nat.moe_dropout_add(o["x"], o["residual"], 0.1, dev(RNG), o["y"], 0)
    else:
        with pytest.raises(ValueError, match="rows"):
            nat.moe_dropout_backward(o["dy"], 0.1, dev(RNG), o["dx"], 0)


def test_dropout_row_strides_that_stay_allowed(nat):
    """Dense, strided and single rows give the library the stride that they have."""
    def shape(t):
        return nat._rows_of("x", dev(t))

    assert shape(torch.zeros(7, 8)) == (7, 8, 8)
    assert shape(torch.zeros(7, 16)[:, :8]) == (7, 8, 16)
    assert shape(torch.zeros(2, 3, 8)) == (6, 8, 8)
    assert shape(torch.zeros(8)) == (1, 8, 8)
    assert shape(torch.zeros(8).expand(1, 8)) == (1, 8, 8)
    assert shape(torch.zeros(7, 3)[:, :1]) == (7, 1, 3)
    assert shape(torch.zeros(0, 8)) == (0, 8, 8)
