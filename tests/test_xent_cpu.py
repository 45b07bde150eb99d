"""What the linear softmax cross entropy refuses before it touches the device, and its workspace's size (no GPU)."""
import pytest
import torch

P = 1 << 20          # an address that nothing reads: every call here is refused first
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lay():
    import __graft_entry__
    __graft_entry__.build()
    from chunkwise_delta_rule_02_gb300 import layers
    return layers


def shape(lay, B=2, T=20, K=16, V=30, dtype=1, ignore=-100):
    return lay._XENT_SHAPE.pack(B, T, K, V, dtype, 0, ignore)


def view(lay, p=P, b=320, t=16):
    return lay._VIEW.pack(p, b, 0, t)


def test_sizes(lay):
    f = lambda s, x=None, w=None, bwd=0: lay._L().dn_xent_workspace_size(s, x or view(lay), w or view(lay, b=0), bwd)  # noqa: E731
    a256 = lambda n: (n + 255) // 256 * 256  # noqa: E731
    M, V = 40, 30
    fwd = f(shape(lay))
    assert lay._XENT_SHAPE.size == 32 and fwd % 256 == 0 and fwd >= 256 + a256(M * 4) + a256(M * 8)
    assert f(shape(lay), bwd=1) == 256 + a256(M * 16 * 2) + a256(M * 256 * 2)      # x is copied: without the tokens that have no target
    assert f(shape(lay, T=100), view(lay, b=1600)) == 256 + a256(200 * 4) + a256(200 * 2 * 8)    # two halves of one tile of the vocabulary
    # rows that do not start at 16 bytes, or at no one distance, are read from a copy
    assert f(shape(lay), view(lay, P + 2)) == fwd + a256(M * 16 * 2) == f(shape(lay), view(lay, b=400)) == f(shape(lay), view(lay, b=340, t=17))
    assert f(shape(lay), None, view(lay, b=0, t=17)) == fwd + a256(V * 16 * 2)
    # float32: three planes of both
    assert f(shape(lay, dtype=0)) == fwd + a256(3 * M * 16 * 2) + a256(3 * V * 16 * 2)
    assert f(shape(lay, B=0)) == 256 == f(shape(lay, T=0))
    # pieces of the vocabulary: the sums of dx are kept between them; dw's long contraction of few tiles is cut
    big = shape(lay, B=1, T=1 << 16, V=5000)
    whole = 256 + (16 * 2 << 16) + (1024 * 2 << 16) + (16 * 4 << 16)
    assert f(big, view(lay, b=0), None, 1) > whole and (f(big, view(lay, b=0), None, 1) - whole) % (1024 * 16 * 4) == 0
    for bad in (dict(B=-1), dict(T=-1), dict(K=0), dict(V=0), dict(dtype=2), dict(B=1 << 20, T=1 << 20), dict(V=(1 << 30) + 1), dict(K=(1 << 24) + 1),
                dict(B=1, T=1 << 30, V=1 << 30)):
        assert f(shape(lay, **bad)) == 0, bad
    assert f(shape(lay), view(lay, P + 1)) == 0 and f(shape(lay), view(lay, 0)) == 0 and f(shape(lay), None, view(lay, 0)) == 0


def test_refusals(lay):
    L, s, v = lay._L(), shape(lay), view(lay)

    def fwd(s=s, x=v, w=v, t=v, loss=P, lse=P, ws=P, n=1 << 20):
        return L.dn_xent_fwd(s, x, w, t, loss, lse, ws, n, None)

    def bwd(s=s, x=v, w=v, t=v, lse=P, dloss=v, dx=v, dw=P, ws=P, n=1 << 20):
        return L.dn_xent_bwd(s, x, w, t, lse, dloss, dx, dw, ws, n, None)

    for call in (fwd, bwd):
        assert call(s=shape(lay, V=0)) == INVALID and call(s=shape(lay, V=(1 << 30) + 1)) == UNSUPPORTED
        for name in ("x", "w", "t"):
            assert call(**{name: None}) == INVALID and call(**{name: view(lay, 0)}) == INVALID and call(**{name: view(lay, P + 1)}) == INVALID
        assert call(lse=None) == INVALID and call(lse=P + 2) == INVALID
        assert call(ws=None) == WORKSPACE and call(ws=P + 8) == WORKSPACE and call(n=256) == WORKSPACE
    assert fwd(loss=None) == INVALID and fwd(loss=P + 1) == INVALID
    for name in ("dloss", "dx"):
        assert bwd(**{name: None}) == INVALID and bwd(**{name: view(lay, P + 1)}) == INVALID
    assert bwd(dw=None) == INVALID and bwd(dw=P + 1) == INVALID


def test_python_refusals_without_a_device(lay):
    x, w, t = torch.zeros(4, 8), torch.zeros(5, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        lay.xent_forward(x, w, t)
    with pytest.raises(ValueError):
        lay.xent_forward(x[0], w, t)
