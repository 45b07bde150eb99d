"""GPU tests of the short causal convolution and of the RMS norm with gate / residual sum against plain
64-bit forms: types, widths, odd sizes, strides, packed sequences with empty and one-token members,
initial and final taps, gradients (against the formula's and against differences), refusals.

Bounds, relative Frobenius per tensor.  A bf16 result is a float32 one rounded once to 8 significant bits:
at most 2^-8 an element, 2^-8 / sqrt(3) / 1.4 = 1.7e-3 over many (errors uniform within half a unit in the
last place, significands spread over [1, 2)); 2^-9 = 1.95e-3 is asked.  float32 results: the sums of the longest case (some 1000 terms,
summed in runs of 64 and then pairwise-like) and the exponential and reciprocal of the sigmoid (a few
2^-22, its argument's rounding included) stay below 5e-6."""
import math

import pytest
import torch

import layers_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = {torch.float32: 5e-6, torch.bfloat16: 2.0 ** -9 + 5e-6}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture()
def gdn():
    import chunkwise_delta_rule_02_gb300 as g
    return g


def close(got, want, dtype=None, scale=1.0):
    e = ref.err(got, want)
    assert e <= scale * TOL[dtype or got.dtype], e


def rnd(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, dtype=F32, scale=1.0: (torch.randn(*s, generator=g) * scale).to(dtype).to(DEV)


def inside(t, pad=3):
    """The same values as a strided view into a larger buffer of NaN: what lies around must not be read."""
    big = torch.full([n + 2 * pad for n in t.shape[:-1]] + [t.shape[-1] + 16], float("nan"), dtype=t.dtype, device=t.device)
    v = big[tuple(slice(pad, pad + n) for n in t.shape[:-1]) + (slice(8, 8 + t.shape[-1]),)]
    v.copy_(t)
    return v


CONV = [  # B, H, T, d, W, dtype, silu, bias, state, lengths
    (2, 3, 70, 128, 4, BF, True, True, False, None),
    (1, 2, 200, 64, 3, F32, True, True, True, None),
    (2, 1, 33, 100, 2, F32, False, False, True, None),
    (1, 3, 129, 129, 4, BF, True, True, True, None),        # odd features: one element an access
    (3, 2, 1, 16, 4, F32, True, True, True, None),          # one token
    (2, 2, 2, 8, 4, BF, True, False, True, None),           # shorter than the taps
    (2, 1, 3, 8, 4, F32, True, True, False, None),
    (1, 2, 140, 128, 4, BF, True, True, True, [0, 1, 70, 0, 2, 64, 3, 0]),
    (1, 1, 131, 40, 3, F32, True, True, False, [64, 1, 66]),
    (1, 2, 67, 12, 2, F32, True, True, True, [67]),
    (2, 2, 0, 16, 4, F32, True, True, True, None),          # no tokens
    (1, 1, 700, 264, 4, BF, True, True, False, None),
]


def conv_case(c, seed=1):
    B, H, T, d, W, dt, act, bias, state, lens = c
    r = rnd(seed)
    n = B if lens is None else len(lens)
    C = H * d
    cu = None if lens is None else torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)
    return dict(x=r(B, H, T, d, dtype=dt), w=r(C, W, scale=W ** -0.5), bias=r(C, scale=0.2) if bias else None,
                state=r(n, W - 1, C, dtype=dt) if state else None, cu=cu, act=act, dy=r(B, H, T, d, dtype=dt),
                dstate=r(n, W - 1, C, dtype=dt))


@pytest.mark.parametrize("c", CONV)
def test_conv_forward(gdn, c):
    k = conv_case(c)
    y, sT = gdn.conv_forward(k["x"], k["w"], k["bias"], k["state"], cu_seqlens=k["cu"], silu=k["act"])
    ry, rs = ref.conv(*(ref.d64(k[n]) for n in ("x", "w", "bias", "state")), cu=k["cu"], act=k["act"])
    close(y, ry)
    assert torch.equal(sT.cpu().double(), rs)      # inputs, moved


@pytest.mark.parametrize("c", CONV)
@pytest.mark.parametrize("upstream_state", [False, True])
def test_conv_backward(gdn, c, upstream_state):
    k = conv_case(c, 2)
    ds = k["dstate"] if upstream_state else None
    g = gdn.conv_backward(k["x"], k["w"], k["bias"], k["state"], k["dy"], ds, cu_seqlens=k["cu"], silu=k["act"])
    leaves = {n: ref.leaf(k[n]) for n in ("x", "w", "bias", "state") if k[n] is not None}
    outs = ref.conv(leaves["x"], leaves["w"], leaves.get("bias"), leaves.get("state"), cu=k["cu"], act=k["act"])
    want = dict(zip(leaves, ref.grads(outs, (ref.d64(k["dy"]), ref.d64(ds)), list(leaves.values()))))
    close(g["dx"], want["x"])
    close(g["dw"], want["w"])
    for name, key in (("dbias", "bias"), ("dstate", "state")):
        if k[key] is None:
            assert g[name] is None
        else:
            close(g[name], want[key])


def test_conv_gradient_against_differences(gdn):
    k = conv_case((1, 2, 37, 24, 4, F32, True, True, True, [5, 0, 1, 31]), 3)
    g = gdn.conv_backward(k["x"], k["w"], k["bias"], k["state"], k["dy"], k["dstate"], cu_seqlens=k["cu"])
    base = {n: ref.d64(k[n]) for n in ("x", "w", "bias", "state")}
    gen = torch.Generator().manual_seed(4)
    for n, got in (("x", g["dx"]), ("w", g["dw"]), ("bias", g["dbias"]), ("state", g["dstate"])):
        way = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        f = []
        for sign in (1, -1):
            a = dict(base, **{n: base[n] + sign * 1e-5 * way})
            y, s = ref.conv(a["x"], a["w"], a["bias"], a["state"], cu=k["cu"])
            f.append(float((y * ref.d64(k["dy"])).sum() + (s * ref.d64(k["dstate"])).sum()))
        diff, dot = (f[0] - f[1]) / 2e-5, float((got.cpu().double() * way).sum())
        # central differences: h^2 ~ 1e-10 and cancellation 1e-16 / 1e-5, both relative to the sum's terms
        size = float((got.cpu().double() * way).abs().sum())
        assert abs(diff - dot) <= 1e-5 * size, (n, diff, dot)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_conv_strides(gdn, dtype):
    """Token-major input, head-major output, slices of wider buffers, a broadcast batch; nothing around is touched."""
    B, H, T, d, W = 2, 3, 50, 64, 4
    r = rnd(5)
    x = inside(r(B, T, H, d, dtype=dtype)).transpose(1, 2)
    w, bias = r(H * d, W), r(H * d)
    out = inside(torch.zeros(B, H, T, d, dtype=dtype, device=DEV))
    y, _ = gdn.conv_forward(x, w, bias, out=out)
    assert y is out
    ry, _ = ref.conv(ref.d64(x), ref.d64(w), ref.d64(bias), None)
    close(y, ry)
    big = out._base
    assert int(torch.isfinite(big).sum()) == out.numel()
    # [B,T,C] is the same with one head
    y3, _ = gdn.conv_forward(x.transpose(1, 2).flatten(2), w, bias)
    assert torch.equal(y3.view(B, T, H, d).transpose(1, 2), y)
    one = r(1, H, T, d, dtype=dtype)
    ye, _ = gdn.conv_forward(one.expand(3, H, T, d), w, bias)
    y1, _ = gdn.conv_forward(one, w, bias)
    assert torch.equal(ye, y1.expand(3, H, T, d))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W,C", [(4, 256), (3, 100), (2, 7)])
def test_conv_step_continues_the_forward(gdn, dtype, W, C):
    """Prefill T tokens, then single tokens: the outputs of one forward over all of them, bit for bit in the taps."""
    N, T, more = 3, 9, 5
    r = rnd(6)
    x, w, bias = r(N, T + more, C, dtype=dtype), r(C, W), r(C)
    y, last = gdn.conv_forward(x, w, bias)
    _, state = gdn.conv_forward(x[:, :T], w, bias)
    for t in range(T, T + more):
        if t % 2:
            got, state = gdn.conv_step(x[:, t], w, bias, state, out_state=state)
        else:
            got, state = gdn.conv_step(x[:, t], w, bias, state)
        close(got, ref.d64(y[:, t]), scale=2.0)      # both sides rounded
    assert torch.equal(state, last)
    got, state = gdn.conv_step(x[:, 0], w, bias, None)
    close(got, ref.d64(y[:, 0]), scale=2.0)


def test_conv_infinities_stay_in_their_channel_and_sequence(gdn):
    r = rnd(7)
    x, w = r(1, 1, 40, 32, dtype=F32), r(32, 4)
    cu = torch.tensor([0, 20, 40], dtype=torch.int32, device=DEV)
    x[0, 0, 18, 5], x[0, 0, 19, 6] = float("inf"), float("nan")
    y, _ = gdn.conv_forward(x, w, cu_seqlens=cu)
    bad = ~torch.isfinite(y[0, 0])
    assert not bad[20:].any() and not bad[:18].any()
    assert set(bad.nonzero()[:, 1].tolist()) <= {5, 6} and bad[18, 5] and bad[19, 6]


def test_conv_malformed_offsets_raise(gdn):
    r = rnd(8)
    x, w = r(1, 1, 40, 32, dtype=F32), r(32, 4)
    for bad in ([0, 30, 20, 40], [0, 20, 41], [1, 20, 40], [0, 20, 39]):
        cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
        with pytest.raises(gdn.GdnError):
            gdn.conv_forward(x, w, cu_seqlens=cu)
        with pytest.raises(gdn.GdnError):
            gdn.conv_backward(x, w, None, None, x, cu_seqlens=cu)


def test_conv_refusals(gdn):
    r = rnd(9)
    x, w = r(2, 3, 10, 16, dtype=BF), r(48, 4)
    for f, e in ((lambda: gdn.conv_forward(x.half(), w), TypeError),
                 (lambda: gdn.conv_forward(x, w.bfloat16()), TypeError),
                 (lambda: gdn.conv_forward(x, w[:40]), ValueError),
                 (lambda: gdn.conv_forward(x, r(48, 5)), gdn.GdnError),
                 (lambda: gdn.conv_forward(x, r(48, 1)), gdn.GdnError),
                 (lambda: gdn.conv_forward(x.transpose(2, 3), r(30, 4)), ValueError),
                 (lambda: gdn.conv_forward(x.cpu(), w), TypeError),
                 (lambda: gdn.conv_forward(x, w, None, r(2, 3, 48)), TypeError),          # taps of another type
                 (lambda: gdn.conv_forward(x, w, None, r(2, 2, 48, dtype=BF)), ValueError),
                 (lambda: gdn.conv_forward(x, w, cu_seqlens=torch.tensor([0, 10], dtype=torch.int32, device=DEV)), ValueError),
                 (lambda: gdn.conv_forward(x[:1], w, cu_seqlens=torch.tensor([0, 10], device=DEV)), TypeError),
                 (lambda: gdn.conv_forward(x, w, out=x[:1].expand(2, 3, 10, 16)), ValueError),
                 (lambda: gdn.conv_step(x[:, 0], w), ValueError),
                 (lambda: gdn.conv_backward(x, w, None, None, x.float()), TypeError)):
        with pytest.raises(e):
            f()


NORM = [  # B, H, T, d, dtype, gate, residual, scale, per head
    (2, 3, 17, 128, BF, True, False, False, False),
    (1, 4, 33, 64, F32, True, False, False, True),
    (2, 1, 9, 2048, BF, False, True, True, False),
    (1, 1, 5, 4096, F32, False, True, False, False),
    (3, 2, 7, 100, F32, True, False, False, False),
    (1, 7, 11, 129, BF, True, False, False, True),          # one element an access
    (1, 1, 3, 2050, BF, False, True, True, False),
    (2, 2, 1, 8, F32, True, True, True, False),
    (1, 1, 1, 1, F32, False, False, False, False),
    (5, 1, 300, 256, BF, False, False, False, False),
    (2, 3, 40, 512, BF, True, True, True, True),
    (1, 1, 2, 16384, F32, False, True, True, False),
    (1, 1, 2, 16383, BF, False, True, True, False),
    (2, 2, 0, 64, F32, True, False, False, False),          # no rows
]


def norm_case(c, seed=1):
    B, H, T, d, dt, gate, res, scale, per = c
    r = rnd(seed)
    s = (B, H, T, d)
    return dict(x=r(*s, dtype=dt), w=r(H, d) if per else r(d), z=r(*s, dtype=dt) if gate else None,
                residual=r(*s, dtype=dt, scale=2.0) if res else None, res_scale=r(d) if scale else None,
                dy=r(*s, dtype=dt), dsum=r(*s, dtype=dt) if res else None)


@pytest.mark.parametrize("c", NORM)
def test_norm_forward(gdn, c):
    k = norm_case(c)
    got = gdn.norm_forward(k["x"], k["w"], z=k["z"], residual=k["residual"], res_scale=k["res_scale"])
    ry, rr = ref.norm(*(ref.d64(k[n]) for n in ("x", "w", "z", "residual", "res_scale")))
    if k["residual"] is None:
        close(got, ry)
    else:
        close(got[0], ry)
        close(got[1], rr)


@pytest.mark.parametrize("c", NORM)
@pytest.mark.parametrize("with_dsum", [False, True])
def test_norm_backward(gdn, c, with_dsum):
    k = norm_case(c, 2)
    res = k["residual"] is not None
    if with_dsum and not res:
        pytest.skip("dsum needs a residual")
    # r is an input of the backward pass: as the forward pass stored it
    total = ref.norm(*(ref.d64(k[n]) for n in ("x", "w", "z", "residual", "res_scale")))[1].to(k["x"].dtype).to(DEV)
    ds = k["dsum"] if with_dsum else None
    g = gdn.norm_backward(k["x"], k["w"], k["dy"], z=k["z"], sum=total if res else None, dsum=ds, res_scale=k["res_scale"])
    names = ["r", "w"] + (["z"] if k["z"] is not None else [])
    leaves = dict(r=ref.leaf(total), w=ref.leaf(k["w"]), z=ref.leaf(k["z"]))
    y, _ = ref.norm(leaves["r"], leaves["w"], leaves["z"])
    want = dict(zip(names, ref.grads((y, leaves["r"]), (ref.d64(k["dy"]), ref.d64(ds)), [leaves[n] for n in names])))
    # dr = q (g - r q^2 mean(g r)): both terms are of g's size, what is left may be smaller (d = 1: nothing is)
    floor = 0.0
    if c[3] == 1:
        floor = float(ref.d64(k["dy"]).norm())
    dr = want["r"]
    scale = 1.0 if k["res_scale"] is None else ref.d64(k["res_scale"])
    tol = TOL[k["x"].dtype]

    def near(got, want):
        e = float((got.cpu().double() - want).norm())
        assert e <= tol * max(float(want.norm()), floor), (e, float(want.norm()))

    near(g["dx"], scale * dr)
    close(g["dw"], want["w"])
    if k["z"] is not None:
        close(g["dz"], want["z"])
    else:
        assert g["dz"] is None
    if res:
        near(g["dresidual"], dr)
    if k["res_scale"] is not None:
        close(g["dres_scale"], (dr * ref.d64(k["x"])).sum((0, 1, 2)))
    else:
        assert g["dres_scale"] is None


def test_norm_gradient_against_differences(gdn):
    k = norm_case((2, 2, 5, 24, F32, True, True, True, True), 3)
    _, r = gdn.norm_forward(k["x"], k["w"], z=k["z"], residual=k["residual"], res_scale=k["res_scale"])
    g = gdn.norm_backward(k["x"], k["w"], k["dy"], z=k["z"], sum=r, dsum=k["dsum"], res_scale=k["res_scale"])
    base = {n: ref.d64(k[n]) for n in ("x", "w", "z", "residual", "res_scale")}
    gen = torch.Generator().manual_seed(4)
    for n, key in (("x", "dx"), ("w", "dw"), ("z", "dz"), ("residual", "dresidual"), ("res_scale", "dres_scale")):
        way = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        f = []
        for sign in (1, -1):
            a = dict(base, **{n: base[n] + sign * 1e-5 * way})
            y, s = ref.norm(*(a[m] for m in ("x", "w", "z", "residual", "res_scale")))
            f.append(float((y * ref.d64(k["dy"])).sum() + (s * ref.d64(k["dsum"])).sum()))
        got = g[key].cpu().double() * way
        assert abs((f[0] - f[1]) / 2e-5 - float(got.sum())) <= 2e-5 * float(got.abs().sum()), n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_strides(gdn, dtype):
    """Head-major rows, token-major gate and result, slices of wider buffers."""
    B, H, T, d = 2, 3, 21, 64
    r = rnd(5)
    x, z = inside(r(B, H, T, d, dtype=dtype)), inside(r(B, T, H, d, dtype=dtype)).transpose(1, 2)
    w = r(d)
    out = inside(torch.zeros(B, T, H, d, dtype=dtype, device=DEV))
    gdn.norm_forward(x, w, z=z, out=out.transpose(1, 2))
    close(out.transpose(1, 2), ref.norm(ref.d64(x), ref.d64(w), ref.d64(z))[0])
    assert int(torch.isfinite(out._base).sum()) == out.numel()
    # rows given as [R,d] and [B,T,d] are the same rows
    xf = r(B, T, d, dtype=dtype)
    a = gdn.norm_forward(xf, w)
    assert torch.equal(a, gdn.norm_forward(xf.view(-1, d), w).view(B, T, d))


def test_norm_rows_are_independent(gdn):
    """A row of zeros gives zeros, one with an infinity or NaN spoils itself alone."""
    r = rnd(6)
    x, w = r(1, 1, 40, 128, dtype=F32), r(128)
    x[0, 0, 3], x[0, 0, 7, 5], x[0, 0, 9, 1] = 0.0, float("inf"), float("nan")
    y = gdn.norm_forward(x, w)
    assert torch.equal(y[0, 0, 3], torch.zeros_like(y[0, 0, 3]))
    bad = (~torch.isfinite(y[0, 0])).any(-1).nonzero()[:, 0].tolist()
    assert set(bad) == {7, 9}


def test_norm_refusals(gdn):
    r = rnd(9)
    x, w = r(2, 3, 10, 16, dtype=BF), r(16)
    for f, e in ((lambda: gdn.norm_forward(x.half(), w), TypeError),
                 (lambda: gdn.norm_forward(x, r(15)), ValueError),
                 (lambda: gdn.norm_forward(x, r(2, 16)), ValueError),
                 (lambda: gdn.norm_forward(x, w, z=x[:1]), ValueError),
                 (lambda: gdn.norm_forward(x, w, z=x.float()), TypeError),
                 (lambda: gdn.norm_forward(x, w, res_scale=w), ValueError),
                 (lambda: gdn.norm_forward(x, w, eps=-1.0), gdn.GdnError),
                 (lambda: gdn.norm_forward(x, w, out=x[:, :, :, ::2]), ValueError),
                 (lambda: gdn.norm_forward(r(1, 1, 1, 16400), r(16400)), gdn.GdnError),
                 (lambda: gdn.norm_backward(x, w, x, dsum=x), ValueError),
                 (lambda: gdn.norm_forward(x.cpu(), w), TypeError)):
        with pytest.raises(e):
            f()


def test_layers_run_on_the_current_stream(gdn):
    """Inputs made on one stream, operators on another that waits for it: the allocations and launches follow."""
    r = rnd(10)
    x, w = r(2, 4, 500, 128, dtype=BF), r(512, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, s = gdn.conv_forward(x, w)
        n = gdn.norm_forward(y, r(128))
    torch.cuda.current_stream().wait_stream(side)
    y0, s0 = gdn.conv_forward(x, w)
    assert torch.equal(y, y0) and torch.equal(s, s0) and math.isfinite(float(n.float().sum()))


def test_backward_sums_repeat_bit_for_bit(gdn):
    k = conv_case((2, 4, 900, 128, 4, BF, True, True, False, None), 11)
    a, b = (gdn.conv_backward(k["x"], k["w"], k["bias"], None, k["dy"]) for _ in range(2))
    n = norm_case((2, 4, 900, 128, BF, True, False, False, False), 12)
    c, d = (gdn.norm_backward(n["x"], n["w"], n["dy"], z=n["z"]) for _ in range(2))
    for p, q in ((a, b), (c, d)):
        for key in p:
            if p[key] is not None:
                assert torch.equal(p[key], q[key]), key
