"""GPU test of the operators together: the hybrid example trains (every parameter has a gradient and the loss
falls), and its single-token path gives the whole sequence's logits."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    import __graft_entry__
    __graft_entry__.build()
    import hybrid_blocks
    return hybrid_blocks


def test_training_lowers_the_loss(ex):
    torch.manual_seed(0)
    model = ex.HybridModel().cuda()
    losses = ex.train(model, steps=12, n=4, T=64)
    assert all(v == v for v in losses)
    assert not [n for n, p in model.named_parameters() if p.grad is None or not bool(torch.isfinite(p.grad).all())]
    assert sum(losses[-3:]) / 3 < 0.9 * losses[0], losses


def test_single_tokens_give_the_sequence(ex):
    torch.manual_seed(1)
    model = ex.HybridModel(pairs=2).cuda()
    tokens = ex.batch(3, 40, 64, torch.Generator().manual_seed(2))
    with torch.no_grad():
        whole = model(tokens).float()
    states = model.start(3)
    single = torch.stack([model.step(tokens[:, t], states).float() for t in range(tokens.shape[1])], 1)
    # bf16 between every two operators, rounded at other places in the two paths: some ten roundings of 2^-8 deep
    assert float((single - whole).norm() / whole.norm()) < 0.04

