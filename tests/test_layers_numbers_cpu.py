"""Numbers that a record of the recurrence, the loss or dropout cannot hold raise ValueError like other arguments (no GPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def lay():
    import __graft_entry__
    __graft_entry__.build()
    from chunkwise_delta_rule_02_gb300 import layers
    return layers


def wide(*shape):
    """A tensor of any sizes, of one element's memory."""
    return torch.zeros(1).expand(shape)


@pytest.mark.parametrize("c", [None, "8"])
def test_recurrence(lay, c):
    with pytest.raises(ValueError):
        lay.recur_shape(torch.zeros(2, 3, 4), c)


@pytest.mark.parametrize("c", [1e39, -1e300])
def test_recurrence_beyond_float32(lay, c):
    """Held as an infinity, which the library refuses."""
    assert lay.dn_recur_workspace_size(lay.recur_shape(torch.zeros(2, 3, 4), c)) == 0


def test_recurrence_sizes(lay):
    with pytest.raises(ValueError):
        lay.recur_shape(wide(2, 1 << 31, 4))
    assert lay.recur_shape(wide(2, 7, 4), 3.5) == lay._RECUR_SHAPE.pack(2, 7, 4, 0, 3.5, 0, 0)


@pytest.mark.parametrize("ignore", [1 << 63, -(1 << 63) - 1, None, 1.5])
def test_loss(lay, ignore):
    with pytest.raises(ValueError):
        lay.xent_shape(torch.zeros(2, 4), torch.zeros(5, 4), ignore)


def test_loss_sizes(lay):
    with pytest.raises(ValueError):
        lay.xent_shape(wide(1 << 31, 4), torch.zeros(5, 4))
    with pytest.raises(ValueError):
        lay.xent_shape(torch.zeros(2, 4), wide(1 << 31, 4))


def test_dropout(lay):
    x = torch.zeros(2, 4)
    for bad in (None, "0.1"):
        with pytest.raises(ValueError):
            lay.dn_dropout(x, bad, x, None, x, 0)
    big = wide(1 << 31, 4)
    with pytest.raises(ValueError):
        lay.dn_dropout(big, 0.1, x, None, big, 0)
