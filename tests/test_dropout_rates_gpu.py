"""GPU tests of dropout at rates next to 1, where a word decides that comes once in 2^32: 0xFFFFFFFF is the first one of seed 7, call
366553561 (found by search, checked here against the generator in Python's integers).  p below 1 - 2^-33 keeps it, times 1 / (1 - p); above,
round(p 2^32) is 2^32, and nothing is kept."""
import pytest
import torch

import recur_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
SEED, CALL = 7, 366553561


@pytest.fixture()
def gdn():
    import __graft_entry__
    __graft_entry__.build()
    import chunkwise_delta_rule_02_gb300 as g
    return g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape,offset", [((1, 1), 0), ((1, 3), 0), ((1, 4), 0), ((1, 64), 0), ((1, 64), 1), ((2, 4, 16), 0)])
def test_the_largest_word(gdn, shape, offset, dtype):
    assert recur_ref.words(SEED, CALL, 1) == [0xFFFFFFFF]
    rng = torch.tensor([SEED, CALL], device=DEV)
    x = torch.ones(2 * torch.Size(shape).numel(), dtype=dtype, device=DEV)[offset:offset + torch.Size(shape).numel()].view(shape)
    for p in (1 - 2.0 ** -20, 1 - 2.0 ** -32):
        y = gdn.dropout_forward(x, p, rng)
        kept = recur_ref.keep(SEED, CALL, p, shape)
        assert bool(kept.flatten()[0]) and torch.equal(y.cpu().double(), torch.where(kept, 1 / (1 - p), 0.0).double())
    r = torch.full_like(x, 3.0)
    for p in (1 - 2.0 ** -34, 1 - 2.0 ** -53):
        assert not bool(recur_ref.keep(SEED, CALL, p, shape).any())
        assert not bool(gdn.dropout_forward(x, p, rng).any()) and not bool(gdn.dropout_backward(x, p, rng).any())
        assert torch.equal(gdn.dropout_forward(x, p, rng, residual=r), r)
        assert not bool(gdn.dropout_forward(torch.full_like(x, float("nan")), p, rng).any())      # what is dropped is not used
