"""GPU test: the single-token calls (residual norm, convolution, scan, gated norm) captured once into a CUDA graph and
replayed give the same bits as the calls themselves, token after token, states updated in place."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("dtype,R,D,N", [(BF, 5, 256, 16), (F32, 1, 100, 7)])
def test_decode_step_in_a_graph(dtype, R, D, N):
    import chunkwise_delta_rule_02_gb300 as gdn
    gen = torch.Generator().manual_seed(5)
    rnd = lambda *s, dt=F32, k=1.0: (torch.randn(*s, generator=gen) * k).to(dt).cuda()
    wn, wg, wc = rnd(D), rnd(D), rnd(D, 4, k=0.5)
    A, bias = -rnd(D, N).abs() - 0.1, rnd(D)
    tokens = [[rnd(R, D, dt=dtype) for _ in range(4)] + [rnd(R, N, dt=dtype) for _ in range(2)] for _ in range(4)]

    def step(tok, taps, h):
        x, res, dt, z, B, C = tok
        y, r = gdn.norm_forward(x, wn, residual=res)
        u, _ = gdn.conv_step(y, wc, None, taps, out_state=taps)
        o, _ = gdn.scan_step(u, dt, A, B, C, None, z, bias, state=h, out_state=h)
        return gdn.norm_forward(o, wg, z=z), r

    def states():
        return torch.zeros(R, 3, D, dtype=dtype, device="cuda"), torch.zeros(R, D, N, device="cuda")

    taps, h = states()
    want = [[t.clone() for t in (step(tok, taps, h)[0], taps, h)] for tok in tokens]

    taps, h = states()
    slot = [t.clone() for t in tokens[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(slot, *states())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(slot, taps, h)[0]
    for tok, w in zip(tokens, want):
        for s, t in zip(slot, tok):
            s.copy_(t)
        graph.replay()
        for got, exp in zip((out, taps, h), w):
            assert torch.equal(got, exp)
