"""GPU tests of dropout: its mask, bit for bit, against the generator in Python's integers; its values against the plain form in
64 bits (a float32 multiplication by 1 / (1 - p), itself rounded, and an addition: 3 x 2^-24 of the operands; bf16 results rounded
once more, 2^-8); strides, odd sizes, the backward pass, replayed graphs, refusals."""
import pytest
import torch

import layers_ref as ref
import recur_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture()
def gdn():
    import chunkwise_delta_rule_02_gb300 as g
    return g


def near(got, want, operands):
    """Within the roundings of float32 (of the operands' size), and of the result's type."""
    step = torch.finfo(got.dtype).eps / 2 if got.dtype != F32 else 0.0
    bound = 3 * 2.0 ** -24 * operands + step * want.abs()
    assert bool(((got.cpu().double() - want).abs() <= bound * (1 + 1e-6)).all())


def rng_of(seed, call):
    return torch.tensor([seed, call], device=DEV)


@pytest.mark.parametrize("shape", [(1, 1), (3, 5), (2, 7, 8), (2, 3, 5, 16), (1, 257, 33), (5, 4, 129), (2, 1, 4099)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("p,seed,call", [(0.1, 0, 0), (0.5, -1, 3), (0.9, 0x123456789ABCDEF, -7), (0.0, 5, 1 << 40)])
def test_values(gdn, shape, dtype, residual, p, seed, call):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(*shape, generator=g).to(dtype).to(DEV)
    r = torch.randn(*shape, generator=g).to(dtype).to(DEV) if residual else None
    y = gdn.dropout_forward(x, p, rng_of(seed, call), residual=r)
    kept = recur_ref.keep(seed, call, p, shape)
    want = recur_ref.dropout(ref.d64(x), p, seed, call, None if r is None else ref.d64(r))
    near(y, want, (ref.d64(x) / (1 - p)).abs() + (0 if r is None else ref.d64(r).abs()))
    if not residual:
        assert torch.equal(y.cpu() != 0, kept & (x.cpu() != 0))
        dx = gdn.dropout_backward(x, p, rng_of(seed, call))
        assert torch.equal(dx, y)


@pytest.mark.parametrize("shape", [(2, 5, 24), (3, 9, 7), (2, 3, 4, 40)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_mask_does_not_go_by_strides(gdn, shape, dtype):
    g = torch.Generator().manual_seed(2)
    x, r = (torch.randn(*shape, generator=g).to(dtype).to(DEV) for _ in range(2))
    rng = rng_of(77, 5)
    want = gdn.dropout_forward(x, 0.3, rng, residual=r)

    def wide(t):
        big = torch.full([n + 1 for n in t.shape[:-1]] + [t.shape[-1] + 24], float("nan"), dtype=dtype, device=DEV)
        v = big[tuple(slice(0, n) for n in t.shape[:-1]) + (slice(16, 16 + t.shape[-1]),)]
        v.copy_(t)
        return v

    def unaligned(t):
        big = torch.full(list(t.shape[:-1]) + [t.shape[-1] + 3], float("nan"), dtype=dtype, device=DEV)
        v = big[..., 1:1 + t.shape[-1]]
        v.copy_(t)
        return v

    turned = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    for f in (wide, unaligned, turned):
        assert torch.equal(gdn.dropout_forward(f(x), 0.3, rng, residual=f(r)), want)
        out = f(torch.zeros_like(x))
        assert gdn.dropout_forward(x, 0.3, rng, residual=f(r), out=out) is out and torch.equal(out, want)
    for which in (0, 1):                    # in place of either input
        a, b = x.clone(), r.clone()
        gdn.dropout_forward(a, 0.3, rng, residual=b, out=(a, b)[which])
        assert torch.equal((a, b)[which], want)
    repeated = x[:1].expand(shape)          # one row for all: the mask is of the whole shape
    assert torch.equal(gdn.dropout_forward(repeated, 0.3, rng), gdn.dropout_forward(repeated.contiguous(), 0.3, rng))


def test_what_is_dropped_is_not_used(gdn):
    x = torch.full((4, 64), float("nan"), device=DEV)
    y = gdn.dropout_forward(x, 0.5, rng_of(3, 4))
    kept = recur_ref.keep(3, 4, 0.5, (4, 64))
    assert torch.equal(torch.isnan(y).cpu(), kept) and bool((y.cpu()[~kept] == 0).all())


def test_how_many_are_kept(gdn):
    """2^22 elements of which each is kept with probability 0.9: the count is within six standard deviations of it."""
    n = 1 << 22
    y = gdn.dropout_forward(torch.ones(n // 64, 64, device=DEV, dtype=BF), 0.1, rng_of(11, 12))
    assert abs(int((y != 0).sum()) - 0.9 * n) <= 6 * (0.09 * n) ** 0.5


def test_a_replayed_graph_draws_what_rng_is_then(gdn):
    x = torch.randn(3, 5, 32, device=DEV)
    rng = rng_of(9, 0)
    gdn.dropout_forward(x, 0.4, rng)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gdn.dropout_forward(x, 0.4, rng)
        dx = gdn.dropout_backward(x, 0.4, rng)
    seen = []
    for call in range(3):
        rng[1] = call
        graph.replay()
        assert torch.equal(y, gdn.dropout_forward(x, 0.4, rng_of(9, call))) and torch.equal(dx, y)
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_no_elements(gdn):
    for shape in ((0, 8), (2, 0, 8), (2, 3, 0)):
        assert gdn.dropout_forward(torch.zeros(shape, device=DEV), 0.1, rng_of(1, 2)).shape == shape


def test_refusals(gdn):
    x, rng = torch.zeros(2, 8, device=DEV), rng_of(1, 2)
    for p in (-0.1, 1.0, float("nan")):
        with pytest.raises(ValueError):
            gdn.dropout_forward(x, p, rng)
    with pytest.raises(TypeError):
        gdn.dropout_forward(x.half(), 0.1, rng)
    with pytest.raises(TypeError):
        gdn.dropout_forward(x, 0.1, rng.int())
    with pytest.raises(TypeError):
        gdn.dropout_forward(x, 0.1, rng.cpu())
    with pytest.raises(ValueError):
        gdn.dropout_forward(x, 0.1, rng[:1])
    with pytest.raises(ValueError):
        gdn.dropout_forward(x[0], 0.1, rng)
    with pytest.raises(ValueError):
        gdn.dropout_forward(x, 0.1, rng, residual=x[:1])
    with pytest.raises(ValueError):
        gdn.dropout_forward(x, 0.1, rng, out=x[:1].expand(2, 8))
