"""GPU tests of the recurrence's single token where a server has it: captured into a graph that is replayed on new tokens with the states
updated in place, and on two streams at once; the bits of the plain calls."""
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


def tokens(n, D, dtype, steps, seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, k=torch.float32: torch.randn(*s, generator=g).to(k).to(DEV)  # noqa: E731
    return dict(rows=[[rnd(n, D, k=dtype) for _ in range(4)] for _ in range(steps)], lam=rnd(D) - 4, bias=[rnd(D), rnd(D)], state=rnd(n, D))


def step(gdn, k, rows, state):
    x, rg, ig, z = rows
    return gdn.recur_step(x, rg, ig, k["lam"], *k["bias"], z=z, state=state, out_state=state)[0]


@pytest.mark.parametrize("n,D,dtype", [(256, 64, torch.bfloat16), (3, 33, torch.bfloat16), (5, 130, torch.float32), (1, 1, torch.float32)])
def test_replayed_from_a_graph(gdn, n, D, dtype):
    k = tokens(n, D, dtype, 6, 1)
    state = k["state"].clone()
    want = [step(gdn, k, rows, state) for rows in k["rows"]]
    slots, held = [t.clone() for t in k["rows"][0]], k["state"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(gdn, k, slots, held)
    held.copy_(k["state"])
    for rows, w in zip(k["rows"], want):
        for s, v in zip(slots, rows):
            s.copy_(v)
        graph.replay()
        assert torch.equal(y, w)
    assert torch.equal(held, state)


def test_two_streams(gdn):
    a, b = (tokens(64, 96, torch.bfloat16, 8, s) for s in (2, 3))
    want = []
    for k in (a, b):
        state = k["state"].clone()
        want.append([step(gdn, k, rows, state) for rows in k["rows"]] + [state])
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    states = [k["state"].clone() for k in (a, b)]
    torch.cuda.synchronize()
    for t in range(8):
        for i, k in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(step(gdn, k, k["rows"][t], states[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(p, q) for p, q in zip(got[i] + [states[i]], want[i]))
