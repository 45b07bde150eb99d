"""GPU tests of the loss at the ends of float32's range: logits of -1e35 and of 1e35, whose largest one is all of lse.  In 64 bits the
others are exp of -1e33 and less, which is 0, and so they are here: lse is a logit, off by the roundings of a sum of 64 terms, 2^-20 of it."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture()
def gdn():
    import __graft_entry__
    __graft_entry__.build()
    import chunkwise_delta_rule_02_gb300 as g
    return g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("M,K", [(2, 64), (2, 576), (40, 64), (300, 64), (300, 67)])
def test_logits_near_the_ends_of_the_range(gdn, M, K, sign, dtype):
    V = 300
    g = torch.Generator().manual_seed(1)
    x = (sign * 1e15 * (1 + torch.rand(M, K, generator=g))).to(dtype).to(DEV)
    w = (1e18 * (1 + torch.arange(V) / 64.0))[:, None].expand(V, K).contiguous().to(dtype).to(DEV)
    t = torch.randint(0, V, (M,), generator=g).to(DEV)
    loss, lse = gdn.xent_forward(x, w, t)
    logits = x.double() @ w.double().t()
    want = torch.logsumexp(logits, 1)
    assert float(want.abs().min()) > 1e34
    room = 2.0 ** -20 * logits.abs().max()
    assert bool(((lse.double() - want).abs() <= room).all())
    assert bool(((loss.double() - (want - logits.gather(1, t[:, None])[:, 0])).abs() <= 2 * room).all())
    g = gdn.xent_backward(x, w, t, lse, torch.full((M,), 1.0 / M, device=DEV))
    assert bool(torch.isfinite(g["dx"]).all()) and bool(torch.isfinite(g["dw"]).all())
