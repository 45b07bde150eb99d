"""GPU tests of loss calls that follow one another without a pause: each kernel of a call may start while the one before it ends, on
the same SMs and with barriers at the same places of shared memory, so that anything still on its way to a block that has left
would reach the next one's.  Expected: the bits of the calls made one at a time."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture()
def gdn():
    import __graft_entry__
    __graft_entry__.build()
    import chunkwise_delta_rule_02_gb300 as g
    return g


def make(M, K, V, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g).to(dtype).to(DEV)
    w = (torch.randn(V, K, generator=g) * 2 * K ** -0.5).to(dtype).to(DEV)
    return x, w, torch.randint(0, V, (M,), generator=g).to(DEV), torch.randn(M, generator=g).to(DEV)


#: few tiles and many, tokens as rows and as columns, one pair of blocks and all of them, short and long contractions, float32 in segments
CALLS = [(300, 64, 500, BF), (20, 128, 700, BF), (257, 16, 257, BF), (100, 512, 20000, BF), (1000, 64, 9000, BF), (40, 48, 300, F32)]


def both(gdn, x, w, t, dloss):
    loss, lse = gdn.xent_forward(x, w, t, check_status=False)
    g = gdn.xent_backward(x, w, t, lse, dloss, check_status=False)
    return loss, lse, g["dx"], g["dw"]


def test_calls_one_after_the_other(gdn):
    inputs = [make(*c, seed=i) for i, c in enumerate(CALLS)]
    want = []
    for k in inputs:
        want.append(both(gdn, *k))
        torch.cuda.synchronize()
    bad = torch.zeros((), dtype=torch.int64, device=DEV)
    for i in range(300):
        n = i * 5 % len(inputs) if i % 2 else i % len(inputs)
        for got, ref in zip(both(gdn, *inputs[n]), want[n]):
            bad += (got != ref).sum()
    assert int(bad) == 0
    for k in inputs:        # and nothing ran out
        _, lse = gdn.xent_forward(*k[:3])
        gdn.xent_backward(*k[:3], lse, k[3])


def test_small_calls_of_one_pair_of_blocks(gdn):
    """One unit a kernel: the blocks leave at once, and the next kernel's may get their SM."""
    k = make(200, 64, 200, BF, 9)
    want = both(gdn, *k)
    torch.cuda.synchronize()
    bad = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(500):
        for got, ref in zip(both(gdn, *k), want):
            bad += (got != ref).sum()
    assert int(bad) == 0
