"""What the library refuses before it touches the device, sizes and records of the gated linear recurrence and of dropout, and the
generator's known answers (no GPU)."""
import ctypes

import pytest
import torch

import recur_ref


@pytest.fixture(scope="module")
def lay():
    import __graft_entry__
    __graft_entry__.build()
    from chunkwise_delta_rule_02_gb300 import layers
    return layers


OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 1 << 20          # an address that nothing reads: every call here is refused first


def shape(lay, B=2, T=20, D=16, dtype=0, c=8.0, n=0, cu=0):
    return lay._RECUR_SHAPE.pack(B, T, D, dtype, c, n, cu)


def io(lay, views=None, pointers=None):
    views = [P] * 5 if views is None else views
    pointers = [P, 0, 0, 0, 0] if pointers is None else pointers
    return lay._RECUR_IO.pack(*[v for p in views for v in (p, 320, 0, 16)], *pointers)


def test_generator_known_answer():
    """Of the method's published vectors: zero key and counter, and all ones."""
    assert recur_ref.words(0, 0, 4) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


def test_records_match_the_header(lay):
    assert lay._RECUR_SHAPE.size == 32 and lay._RECUR_IO.size == 5 * 32 + 5 * 8 and lay._DROPOUT_SHAPE.size == 32


def test_sizes(lay):
    f = lay.dn_recur_workspace_size
    assert f(shape(lay)) == 256 and f(shape(lay), True) > 256
    assert f(shape(lay, B=1, n=3, cu=P)) == 512
    assert lay.dn_recur_saved_size(shape(lay)) == 2 * 3 * 16 * 4
    assert lay.dn_recur_saved_size(shape(lay, T=0)) == 256
    for bad in (dict(B=0), dict(D=0), dict(T=-1), dict(dtype=2), dict(c=-1.0), dict(c=float("nan")), dict(T=(1 << 30) + 1), dict(D=(1 << 24) + 1),
                dict(n=3, cu=P), dict(B=1, n=-1, cu=P), dict(B=1, n=3, cu=P + 2), dict(B=1 << 28)):
        assert f(shape(lay, **bad)) == 0 and lay.dn_recur_saved_size(shape(lay, **bad)) == 0, bad


def test_recur_refusals(lay):
    L = lay._L()
    s, good = shape(lay), io(lay)
    fwd = lambda s, i, saved=None, n=0, ws=P, m=1 << 20: L.dn_recur_fwd(s, i, saved, n, ws, m, None)  # noqa: E731
    assert fwd(shape(lay, D=0), good) == INVALID
    assert fwd(shape(lay, T=(1 << 30) + 1), good) == UNSUPPORTED
    for k in (0, 1, 2, 4):
        assert fwd(s, io(lay, [0 if j == k else P for j in range(5)])) == INVALID      # a missing array
    for k in range(5):
        assert fwd(s, io(lay, [P + 2 if j == k else P for j in range(5)])) == INVALID  # alignment
        assert fwd(s, io(lay, None, [P + 2 if j == k else P for j in range(5)])) == INVALID
    assert fwd(s, io(lay, None, [0, 0, 0, 0, 0])) == INVALID
    assert fwd(s, good, ws=None) == WORKSPACE and fwd(s, good, ws=P + 8) == WORKSPACE and fwd(s, good, m=255) == WORKSPACE
    assert fwd(s, good, P, 383) == WORKSPACE and fwd(s, good, P + 4, 1 << 20) == WORKSPACE
    bwd = lambda g, saved=P, n=384, ws=P, m=1 << 20: L.dn_recur_bwd(s, good, g, saved, n, ws, m, None)  # noqa: E731
    grads = lambda views=None, pointers=(0, P, 0, 0, 0): io(lay, views, list(pointers))  # noqa: E731
    for k in range(5):
        assert bwd(grads([0 if j == k else P for j in range(5)])) == INVALID
        assert bwd(grads([P + 1 if j == k else P for j in range(5)])) == INVALID
    assert bwd(grads(pointers=(0, 0, 0, 0, 0))) == INVALID
    assert bwd(grads(), saved=None) == WORKSPACE and bwd(grads(), n=383) == WORKSPACE and bwd(grads(), m=256) == WORKSPACE
    assert L.dn_recur_step(s, good, None) == INVALID                                   # more than one token
    assert L.dn_recur_step(shape(lay, B=1, T=1, n=1, cu=P), good, None) == INVALID


def test_dropout_refusals(lay):
    L = lay._L()
    view = lay._VIEW.pack(P, 0, 0, 16)

    def call(B=1, H=1, T=4, d=16, dtype=0, p=0.1, x=view, r=None, rng=P, y=view):
        return L.dn_dropout(lay._DROPOUT_SHAPE.pack(B, H, T, d, dtype, 0, p), x, r, rng, y, None)

    for bad in (dict(p=1.0), dict(p=-0.5), dict(p=float("nan")), dict(d=0), dict(H=0), dict(T=-1), dict(B=-1), dict(dtype=2), dict(rng=None),
                dict(rng=P + 4), dict(x=None), dict(y=None), dict(x=lay._VIEW.pack(P + 2, 0, 0, 16)), dict(r=lay._VIEW.pack(P + 2, 0, 0, 16)),
                dict(y=lay._VIEW.pack(P + 1, 0, 0, 16))):
        assert call(**bad) == INVALID, bad
    assert call(B=2 ** 31 - 1, H=2 ** 31 - 1, T=2) == UNSUPPORTED
    assert call(T=0) == OK


def test_python_refusals_without_a_device(lay):
    x = torch.zeros(1, 4, 8)
    with pytest.raises(TypeError):
        lay.recur_forward(x, x, x, torch.zeros(8))
    with pytest.raises(TypeError):
        lay.dropout_forward(x, 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        lay.recur_step(x, x, x, torch.zeros(8))
    assert ctypes.sizeof(ctypes.c_int64) == 8
