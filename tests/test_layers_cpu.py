"""Host-side checks of the layer operators that need no GPU: records as the header lays them out, workspace
and buffer sizes, and every refusal of a C entry point before it touches the device; argument checks of the
Python calls; the plain 64-bit forms of the tests against differences and against the plain forms in
perf/operators.py."""
import ctypes
import importlib.util
import os

import pytest
import torch

import layers_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20          # an address that is never read


@pytest.fixture(scope="module")
def lay():
    import __graft_entry__
    __graft_entry__.build()
    from chunkwise_delta_rule_02_gb300 import layers
    layers._L()
    return layers


def view(lay, p=P, b=0, h=0, t=0):
    return lay._VIEW.pack(p, b, h, t)


def conv(lay, B=2, H=3, T=10, d=16, W=4, dt=1, silu=1, n=0, cu=0):
    return lay._CONV_SHAPE.pack(B, H, T, d, W, dt, silu, n, cu)


def scan(lay, B=2, T=10, D=32, N=16, G=1, dt=1, sp=1, n=0, cu=0):
    return lay._SCAN_SHAPE.pack(B, T, D, N, G, dt, sp, n, cu)


def norm(lay, B=2, H=3, T=10, d=16, dt=1, per=0, eps=1e-6):
    return lay._NORM_SHAPE.pack(B, H, T, d, dt, per, eps, 0)


def io(lay, **over):
    """dn_scan_io of fake addresses; a view or pointer by name replaced."""
    v = dict(x=(P, 320, 0, 32), dt=(P, 320, 0, 32), b=(P, 160, 0, 16), c=(P, 160, 0, 16), z=(0, 0, 0, 0), y=(P, 320, 0, 32),
             A=P, D=P, bias=P, h0=0, hT=0)
    v.update(over)
    return lay._SCAN_IO.pack(*(sum((v[k] for k in ("x", "dt", "b", "c", "z", "y")), ())), v["A"], v["D"], v["bias"], v["h0"], v["hT"])


def grads(lay, **over):
    v = dict(dy=(P, 320, 0, 32), dx=(P, 320, 0, 32), ddt=(P, 320, 0, 32), db=(P, 160, 0, 16), dc=(P, 160, 0, 16), dz=(0, 0, 0, 0),
             dhT=0, dA=P, dD=0, bias=0, dh0=0)
    v.update(over)
    return lay._SCAN_IO.pack(*(sum((v[k] for k in ("dy", "dx", "ddt", "db", "dc", "dz")), ())), v["dhT"], v["dA"], v["dD"], v["bias"], v["dh0"])


def test_records_have_the_header_sizes(lay):
    # dn_view: a pointer and three int64; dn_conv_shape, dn_scan_shape: eight int32 and a pointer
    assert lay._VIEW.size == 32 and lay._CONV_SHAPE.size == 40 and lay._SCAN_SHAPE.size == 40
    assert lay._NORM_SHAPE.size == 32 and lay._SCAN_IO.size == 6 * 32 + 5 * 8


def test_library_exports_the_layer_calls(lay):
    L = ctypes.CDLL(lay.binding.library_path())
    for name in lay.EXPORTS:
        assert hasattr(L, name), name


def test_workspace_sizes(lay):
    assert 0 < lay.dn_conv_workspace_size(conv(lay)) < lay.dn_conv_workspace_size(conv(lay), True)
    assert lay.dn_conv_workspace_size(conv(lay, B=1, n=3, cu=16)) > lay.dn_conv_workspace_size(conv(lay, B=1))
    for bad in (dict(B=0), dict(H=0), dict(T=-1), dict(d=0), dict(dt=2), dict(W=1), dict(W=5), dict(cu=16, n=3), dict(B=1, cu=18, n=3),
                dict(B=1, cu=16, n=-1)):
        assert lay.dn_conv_workspace_size(conv(lay, **bad)) == 0, bad
    assert 0 < lay.dn_scan_workspace_size(scan(lay)) < lay.dn_scan_workspace_size(scan(lay), True)
    # the state before every 8th token up to 32 states (padded to 8, 16, 32), every 16th above
    assert lay.dn_scan_saved_size(scan(lay, B=1, T=17, D=3, N=16)) == 3 * 3 * 16 * 4
    assert lay.dn_scan_saved_size(scan(lay, B=1, T=17, D=3, N=5)) == 3 * 3 * 8 * 4
    assert lay.dn_scan_saved_size(scan(lay, B=2, T=17, D=3, N=33)) == 2 * 2 * 3 * 64 * 4
    for bad in (dict(B=0), dict(T=-1), dict(D=0), dict(N=0), dict(N=129), dict(G=0), dict(G=3), dict(dt=7), dict(cu=16, n=2)):
        assert lay.dn_scan_workspace_size(scan(lay, **bad)) == 0, bad
        assert lay.dn_scan_saved_size(scan(lay, **bad)) == 0, bad
    assert lay.dn_norm_workspace_size(norm(lay)) > 0
    for bad in (dict(B=0), dict(d=0), dict(d=16385), dict(dt=3), dict(eps=-1.0), dict(eps=float("nan"))):
        assert lay.dn_norm_workspace_size(norm(lay, **bad)) == 0, bad


def test_conv_refusals_on_the_host(lay):
    L, b = lay._L(), lay.binding
    v, s = view(lay), conv(lay)
    big = 1 << 40
    assert L.dn_conv_fwd(None, v, P, P, None, v, None, P, big, None) == b.DN_ERR_INVALID_ARG
    assert L.dn_conv_fwd(s, None, P, P, None, v, None, P, big, None) == b.DN_ERR_INVALID_ARG
    assert L.dn_conv_fwd(s, view(lay, 0), P, P, None, v, None, P, big, None) == b.DN_ERR_INVALID_ARG
    assert L.dn_conv_fwd(s, v, None, P, None, v, None, P, big, None) == b.DN_ERR_INVALID_ARG
    assert L.dn_conv_fwd(s, view(lay, P + 1), P, P, None, v, None, P, big, None) == b.DN_ERR_INVALID_ARG
    assert L.dn_conv_fwd(s, v, P + 2, P, None, v, None, P, big, None) == b.DN_ERR_INVALID_ARG
    assert L.dn_conv_fwd(s, v, P, P, None, v, None, None, big, None) == b.DN_ERR_WORKSPACE
    assert L.dn_conv_fwd(s, v, P, P, None, v, None, P, 8, None) == b.DN_ERR_WORKSPACE
    assert L.dn_conv_fwd(conv(lay, W=5), v, P, P, None, v, None, P, big, None) == b.DN_ERR_UNSUPPORTED
    assert L.dn_conv_bwd(s, v, P, P, None, v, None, v, None, P, None, P, big, None) == b.DN_ERR_INVALID_ARG     # no dw
    assert L.dn_conv_bwd(s, v, P, P, None, None, None, v, P, P, None, P, big, None) == b.DN_ERR_INVALID_ARG     # no dy
    assert L.dn_conv_bwd(s, v, P, P, None, v, None, v, P, P, None, P, 256, None) == b.DN_ERR_WORKSPACE
    assert L.dn_conv_step(s, v, P, P, P, P, v, None) == b.DN_ERR_INVALID_ARG                                    # T != 1
    assert L.dn_conv_step(conv(lay, B=1, T=1, cu=16, n=1), v, P, P, P, P, v, None) == b.DN_ERR_INVALID_ARG      # packed
    assert L.dn_conv_step(conv(lay, T=1), v, P, P, P, P, None, None) == b.DN_ERR_INVALID_ARG


def test_scan_refusals_on_the_host(lay):
    L, b = lay._L(), lay.binding
    s, ok, big = scan(lay), io(lay), 1 << 40
    assert L.dn_scan_fwd(None, ok, None, 0, P, big, None) == b.DN_ERR_INVALID_ARG
    assert L.dn_scan_fwd(s, None, None, 0, P, big, None) == b.DN_ERR_INVALID_ARG
    for bad in (dict(A=0), dict(x=(0, 0, 0, 0)), dict(dt=(P + 1, 320, 0, 32)), dict(b=(0, 0, 0, 0)), dict(y=(0, 0, 0, 0)), dict(h0=P + 2)):
        assert L.dn_scan_fwd(s, io(lay, **bad), None, 0, P, big, None) == b.DN_ERR_INVALID_ARG, bad
    assert L.dn_scan_fwd(s, ok, None, 0, None, big, None) == b.DN_ERR_WORKSPACE
    assert L.dn_scan_fwd(s, ok, P, 16, P, big, None) == b.DN_ERR_WORKSPACE                                      # saved too small
    assert L.dn_scan_fwd(scan(lay, N=200), ok, None, 0, P, big, None) == b.DN_ERR_UNSUPPORTED
    g = grads(lay)
    assert L.dn_scan_bwd(s, ok, None, P, big, P, big, None) == b.DN_ERR_INVALID_ARG
    for bad in (dict(dA=0), dict(dy=(0, 0, 0, 0)), dict(dc=(0, 0, 0, 0)), dict(dx=(P + 1, 320, 0, 32)), dict(dhT=P + 1)):
        assert L.dn_scan_bwd(s, ok, grads(lay, **bad), P, big, P, big, None) == b.DN_ERR_INVALID_ARG, bad
    gated = io(lay, z=(P, 320, 0, 32))
    assert L.dn_scan_bwd(s, gated, g, P, big, P, big, None) == b.DN_ERR_INVALID_ARG                             # z without dz
    assert L.dn_scan_bwd(s, ok, g, None, big, P, big, None) == b.DN_ERR_WORKSPACE
    assert L.dn_scan_bwd(s, ok, g, P, big, P, 64, None) == b.DN_ERR_WORKSPACE
    assert L.dn_scan_step(s, ok, None) == b.DN_ERR_INVALID_ARG                                                  # T != 1
    assert L.dn_scan_step(scan(lay, B=1, T=1, cu=16, n=1), ok, None) == b.DN_ERR_INVALID_ARG


def test_norm_refusals_on_the_host(lay):
    L, b = lay._L(), lay.binding
    s, v, big = norm(lay), view(lay), 1 << 40
    assert L.dn_norm_fwd(None, v, P, None, None, None, v, None, None) == b.DN_ERR_INVALID_ARG
    assert L.dn_norm_fwd(s, v, None, None, None, None, v, None, None) == b.DN_ERR_INVALID_ARG
    assert L.dn_norm_fwd(s, v, P, None, None, P, v, None, None) == b.DN_ERR_INVALID_ARG                         # scale, no residual
    assert L.dn_norm_fwd(s, v, P, None, None, None, v, v, None) == b.DN_ERR_INVALID_ARG                         # sum, no residual
    assert L.dn_norm_fwd(s, view(lay, P + 1), P, None, None, None, v, None, None) == b.DN_ERR_INVALID_ARG
    assert L.dn_norm_fwd(norm(lay, d=20000), v, P, None, None, None, v, None, None) == b.DN_ERR_UNSUPPORTED
    bwd = lambda *a: L.dn_norm_bwd(s, *a, P, big, None)  # noqa: E731
    #            x  w  z     scale  sum   dy dsum  dx dw  dz    dres  dscale
    assert bwd(v, P, None, None, None, v, None, v, None, None, None, None) == b.DN_ERR_INVALID_ARG             # no dw
    assert bwd(v, P, None, P, None, v, None, v, P, None, None, None) == b.DN_ERR_INVALID_ARG                   # scale, no sum
    assert bwd(v, P, None, None, None, v, v, v, P, None, None, None) == b.DN_ERR_INVALID_ARG                   # dsum, no sum
    assert bwd(v, P, None, None, None, v, None, v, P, v, None, None) == b.DN_ERR_INVALID_ARG                   # dz, no z
    assert bwd(v, P, None, None, None, v, None, None, P, None, None, None) == b.DN_ERR_INVALID_ARG             # no dx
    assert L.dn_norm_bwd(s, v, P, None, None, None, v, None, v, P, None, None, None, P, 16, None) == b.DN_ERR_WORKSPACE


def test_python_calls_refuse_cpu_tensors_and_wrong_shapes(lay):
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    with pytest.raises(TypeError):
        lay.conv_forward(x, w)
    with pytest.raises(TypeError):
        lay.conv_step(x[:, 0], w)
    with pytest.raises(ValueError):
        lay.conv_forward(x[0], w)
    with pytest.raises(TypeError):
        lay.norm_forward(x, torch.ones(8))
    with pytest.raises(TypeError):
        lay.scan_forward(x, x, -torch.ones(8, 4), torch.zeros(2, 5, 4), torch.zeros(2, 5, 4))
    with pytest.raises(ValueError):
        lay.scan_forward(x, x, -torch.ones(8), torch.zeros(2, 5, 4), torch.zeros(2, 5, 4))


def _plain():
    spec = importlib.util.spec_from_file_location("operators", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.DEV = "cpu"
    return m


@pytest.mark.parametrize("case", [
    dict(op="conv_bwd", type="f32", B=1, H=2, T=17, d=5, W=3, silu=True, packed=5, state=True),
    dict(op="conv_step", type="f32", B=3, H=2, T=1, d=5, W=4, silu=True, packed=0, state=True),
    dict(op="scan_train", type="f32", B=1, T=23, D=6, N=4, G=1, packed=5, state=True, gate=False),
    dict(op="scan_train", type="f32", B=2, T=23, D=6, N=4, G=2, packed=0, state=False, gate=True),
    dict(op="norm_bwd", type="f32", B=2, H=3, T=4, d=5, gate=True, residual=False),
    dict(op="norm_bwd", type="f32", B=2, H=1, T=4, d=5, gate=False, residual=True)])
def test_plain_forms_agree_with_their_64_bit_definitions(case):
    m = _plain()
    got, want = m.run(m.prepare(case, 3)), m.exact(case, 3)
    assert set(got) == set(want)
    for k in want:
        assert (got[k] is None) == (want[k] is None), k
        if want[k] is not None:
            # float32 sums of at most some hundred terms
            assert ref.err(got[k], want[k]) <= 2e-6, k


def test_reference_scan_gradient_against_differences():
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    v = dict(x=r(1, 9, 4), dt=r(1, 9, 4), A=-r(4, 3).abs(), Bm=r(1, 9, 2, 3), Cm=r(1, 9, 2, 3), D=r(4), z=r(1, 9, 4), dt_bias=r(4), h0=r(2, 4, 3))
    cu, dy, dh = [0, 4, 9], r(1, 9, 4), r(2, 4, 3)
    leaves = {k: t.clone().requires_grad_(True) for k, t in v.items()}
    got = dict(zip(v, ref.grads(ref.scan(**leaves, cu=cu), (dy, dh), list(leaves.values()))))
    for k in v:
        way = r(*v[k].shape)
        f = []
        for sign in (1, -1):
            y, h = ref.scan(**dict(v, **{k: v[k] + sign * 1e-6 * way}), cu=cu)
            f.append(float((y * dy).sum() + (h * dh).sum()))
        assert abs((f[0] - f[1]) / 2e-6 - float((got[k] * way).sum())) < 1e-6 * float((got[k] * way).abs().sum() + 1), k
