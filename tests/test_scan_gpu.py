"""GPU tests of the selective state space scan against a plain 64-bit recurrence: types, state counts,
groups, odd sizes, strides, packed sequences with empty and one-token members, initial and final
states, time segments, gradients (against the formula's and against differences), single tokens,
refusals.

Bounds, relative Frobenius per tensor.  bf16 results are float32 ones rounded once to 8 significant
bits: half a unit in the last place, 2^-8 of an element at most, so of the norm.  float32: a
decay is an exponential good to about 2^-22 whose argument is rounded twice (2^-23 of an argument of
order 1); a state remembers 1 / (1 - a) tokens, so it is off by at most that memory times 2^-22 where
all errors agree in sign.  Steps here are about 0.02 .. 1 against A = -1 and below: a memory of at most
50 tokens, 1.2e-5 at the very worst and a tenth of that where the signs vary as they do: 4e-6."""
import pytest
import torch

import layers_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 4e-6, BF: 2.0 ** -8 + 4e-6}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture()
def gdn():
    import chunkwise_delta_rule_02_gb300 as g
    return g


def close(got, want):
    e = ref.err(got, want)
    assert e <= TOL[got.dtype], e


CASES = [  # B, T, D, N, G, dtype, gate, state, skip, bias, softplus, lengths
    (2, 40, 64, 16, 1, F32, True, True, True, True, True, None),
    (1, 33, 100, 16, 1, BF, True, False, True, True, True, None),
    (2, 17, 70, 8, 2, F32, False, True, True, True, True, None),
    (1, 16, 300, 4, 1, F32, True, False, False, False, True, None),
    (1, 31, 130, 3, 1, BF, True, True, True, True, True, None),
    (1, 35, 48, 32, 2, F32, True, True, True, True, True, None),
    (1, 18, 40, 64, 1, BF, False, True, True, False, True, None),
    (1, 19, 20, 100, 1, F32, True, True, True, True, True, None),
    (1, 21, 18, 128, 2, F32, True, False, True, True, True, None),
    (2, 1, 64, 16, 1, F32, True, True, True, True, True, None),              # one token
    (1, 300, 40, 16, 1, F32, True, True, True, True, True, None),            # several time segments
    (1, 700, 20, 5, 1, BF, True, True, True, True, True, None),
    (1, 60, 68, 16, 1, F32, True, True, True, True, True, [0, 1, 30, 0, 2, 16, 11, 0]),
    (1, 400, 12, 16, 1, F32, False, False, True, True, True, [150, 1, 249]),
    (1, 300, 24, 1, 3, BF, True, True, True, True, True, [300]),
    (2, 24, 33, 16, 1, F32, True, True, True, True, False, None),            # steps given as they are
    (2, 0, 32, 16, 1, F32, True, True, True, True, True, None),              # no tokens
]


def make(c, seed=1):
    B, T, D, N, G, dt, gate, state, skip, bias, softplus, lens = c
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, scale=1.0, dtype=F32: (torch.randn(*s, generator=g) * scale).to(dtype).to(DEV)  # noqa: E731
    n = B if lens is None else len(lens)
    cu = None if lens is None else torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)
    k = dict(x=r(B, T, D, dtype=dt), dt=r(B, T, D, scale=0.7, dtype=dt), A=-(0.5 + torch.rand(D, N, generator=g) * 4).to(DEV),
             B=r(B, T, G, N, dtype=dt), C=r(B, T, G, N, dtype=dt), D=r(D) if skip else None,
             z=r(B, T, D, dtype=dt) if gate else None, dt_bias=(r(D, scale=0.3) - 1.5) if bias else None,
             h0=r(n, D, N, scale=0.5) if state else None)
    if not softplus:
        k["dt"] = k["dt"].abs() * 0.2
        k["dt_bias"] = k["dt_bias"].abs() * 0.1
    return k, cu, softplus, r(B, T, D, dtype=dt), r(n, D, N, scale=0.5)


def want_forward(k, cu, softplus):
    v = {n: ref.d64(t) for n, t in k.items()}
    return ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"], v["h0"], cu=cu, softplus=softplus)


@pytest.mark.parametrize("c", CASES)
def test_scan_forward(gdn, c):
    k, cu, softplus, _, _ = make(c)
    y, hT = gdn.scan_forward(**k, cu_seqlens=cu, dt_softplus=softplus)
    ry, rh = want_forward(k, cu, softplus)
    close(y, ry)
    close(hT, rh)


@pytest.mark.parametrize("c", CASES)
@pytest.mark.parametrize("upstream_state", [False, True])
def test_scan_backward(gdn, c, upstream_state):
    k, cu, softplus, dy, dhT = make(c, 2)
    dhT = dhT if upstream_state else None
    y, hT, saved = gdn.scan_forward(**k, cu_seqlens=cu, dt_softplus=softplus, save=True)
    y2, hT2 = gdn.scan_forward(**k, cu_seqlens=cu, dt_softplus=softplus)
    assert torch.equal(y, y2) and torch.equal(hT, hT2)      # keeping the states changes nothing
    g = gdn.scan_backward(**k, dy=dy, dhT=dhT, saved=saved, cu_seqlens=cu, dt_softplus=softplus)
    names = [n for n in k if k[n] is not None]
    v = {n: ref.leaf(k[n]) for n in k}
    outs = ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"], v["h0"], cu=cu, softplus=softplus)
    want = dict(zip(names, ref.grads(outs, (ref.d64(dy), ref.d64(dhT)), [v[n] for n in names])))
    for n in k:
        got = g["d" + n]
        if k[n] is None:
            assert got is None
        else:
            assert got.dtype == k[n].dtype
            # sums over tokens and channels of terms of both signs: what they cancel stays as error
            assert ref.err(got, want[n]) <= (4 if n in ("A", "dt_bias", "dt", "h0") and got.dtype == F32 else 1) * TOL[got.dtype], n


def test_scan_gradient_against_differences(gdn):
    k, cu, softplus, dy, dhT = make((1, 30, 10, 6, 2, F32, True, True, True, True, True, [9, 0, 1, 20]), 3)
    _, _, saved = gdn.scan_forward(**k, cu_seqlens=cu, save=True)
    g = gdn.scan_backward(**k, dy=dy, dhT=dhT, saved=saved, cu_seqlens=cu)
    base = {n: ref.d64(t) for n, t in k.items()}
    gen = torch.Generator().manual_seed(4)
    for n in base:
        way = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)
        f = []
        for sign in (1, -1):
            a = dict(base, **{n: base[n] + sign * 1e-5 * way})
            y, h = ref.scan(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"], a["dt_bias"], a["h0"], cu=cu)
            f.append(float((y * ref.d64(dy)).sum() + (h * ref.d64(dhT)).sum()))
        got = g["d" + n].cpu().double() * way
        assert abs((f[0] - f[1]) / 2e-5 - float(got.sum())) <= 2e-5 * float(got.abs().sum()), n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_strides(gdn, dtype):
    """x and z halves of one projection, B and C cut from another at odd offsets: the results of dense copies."""
    B, T, D, N = 2, 50, 72, 16
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)  # noqa: E731
    xz, low = r(B, T, 2 * D), r(B, T, 5 + 2 * N + 3)
    x, z, Bm, Cm = xz[..., :D], xz[..., D:], low[..., 5:5 + N], low[..., 5 + N:5 + 2 * N]
    dt = r(T, B, D).transpose(0, 1)
    A, skip = -torch.rand(D, N, generator=g).to(DEV) - 0.5, torch.ones(D, device=DEV)
    out = torch.full((B, T, D + 8), float("nan"), dtype=dtype, device=DEV)
    args = (x, dt, A, Bm, Cm, skip, z)
    dense = tuple(t.contiguous() for t in args)
    y, hT, saved = gdn.scan_forward(*args, out=out[..., 4:4 + D], save=True)
    y2, hT2, saved2 = gdn.scan_forward(*dense, save=True)
    assert torch.equal(y, y2) and torch.equal(hT, hT2)
    assert int(torch.isfinite(out).sum()) == y.numel()
    dy = r(T, B, D).transpose(0, 1)
    ga, gb = gdn.scan_backward(*args, dy=dy, saved=saved), gdn.scan_backward(*dense, dy=dy.contiguous(), saved=saved2)
    for n in ga:
        if ga[n] is not None:
            assert torch.equal(ga[n], gb[n]), n


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,N,G", [(64, 16, 1), (30, 5, 2), (24, 100, 1), (8, 1, 1), (40, 128, 1)])
def test_scan_step_continues_the_forward(gdn, dtype, D, N, G):
    n, T, more = 3, 20, 4
    k, _, _, _, _ = make((n, T + more, D, N, G, dtype, True, True, True, True, True, None), 6)
    y, last = gdn.scan_forward(**k)
    pre = {m: (t[:, :T] if m in ("x", "dt", "B", "C", "z") else t) for m, t in k.items()}
    _, state = gdn.scan_forward(**pre)
    for t in range(T, T + more):
        tok = {m: (v[:, t] if m in ("x", "dt", "B", "C", "z") else v) for m, v in k.items() if m != "h0"}
        got, state = gdn.scan_step(**tok, state=state, out_state=state if t % 2 else None)
        e = ref.err(got, ref.d64(y[:, t]))
        assert e <= 2 * TOL[dtype], e
    assert ref.err(state, ref.d64(last)) <= 2 * TOL[F32]
    tok = {m: (v[:, 0] if m in ("x", "dt", "B", "C", "z") else v) for m, v in k.items() if m != "h0"}
    got, state = gdn.scan_step(**tok)
    ry, rh = want_forward({**{m: (v[:, :1] if m in ("x", "dt", "B", "C", "z") else v) for m, v in k.items()}, "h0": None}, None, True)
    close(got, ry[:, 0])
    close(state, rh)


def test_scan_extreme_values(gdn):
    """A step so large that the decay underflows, one of softplus(-100), padded sequences' infinities: nothing leaks."""
    k, _, _, _, _ = make((1, 48, 40, 16, 1, F32, False, True, True, True, True, None), 7)
    k["dt"][0, 5], k["dt"][0, 9] = 100.0, -100.0
    y, h = gdn.scan_forward(**k)
    ry, rh = want_forward(k, None, True)
    close(y, ry)
    close(h, rh)
    cu = torch.tensor([0, 20, 48], dtype=torch.int32, device=DEV)
    k2 = dict(k, h0=k["h0"].expand(2, -1, -1).contiguous())
    clean = gdn.scan_forward(**k2, cu_seqlens=cu, save=True)
    k2["x"] = k2["x"].clone()
    k2["x"][0, 18, 3] = float("inf")
    k2["x"][0, 19, 4] = float("nan")
    dirty = gdn.scan_forward(**k2, cu_seqlens=cu, save=True)
    assert torch.equal(clean[0][0, 20:], dirty[0][0, 20:]) and torch.equal(clean[1][1], dirty[1][1])
    assert torch.equal(clean[0][0, :18], dirty[0][0, :18]) and not torch.isfinite(dirty[1][0, 3]).any()


def test_scan_malformed_offsets_raise(gdn):
    k, _, _, dy, _ = make((1, 40, 32, 16, 1, F32, True, False, True, True, True, None), 8)
    for bad in ([0, 30, 20, 40], [0, 20, 41], [1, 20, 40], [0, 20, 39]):
        cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
        with pytest.raises(gdn.GdnError):
            gdn.scan_forward(**k, cu_seqlens=cu)
        _, _, saved = gdn.scan_forward(**k, cu_seqlens=cu, save=True, check_status=False)
        with pytest.raises(gdn.GdnError):
            gdn.scan_backward(**k, dy=dy, saved=saved, cu_seqlens=cu)


def test_scan_backward_repeats_bit_for_bit(gdn):
    k, cu, _, dy, dhT = make((2, 500, 136, 16, 1, BF, True, True, True, True, True, None), 9)
    _, _, saved = gdn.scan_forward(**k, save=True)
    a, b = (gdn.scan_backward(**k, dy=dy, dhT=dhT, saved=saved) for _ in range(2))
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_scan_refusals(gdn):
    k, _, _, dy, _ = make((2, 10, 32, 16, 1, BF, True, True, True, True, True, None), 10)
    y, hT, saved = gdn.scan_forward(**k, save=True)
    bad = lambda **e: (lambda: gdn.scan_forward(**dict(k, **e)))  # noqa: E731
    cu = torch.tensor([0, 10], dtype=torch.int32, device=DEV)
    for f, e in ((bad(x=k["x"].half()), TypeError), (bad(dt=k["dt"].float()), TypeError), (bad(A=k["A"].bfloat16()), TypeError),
                 (bad(B=k["B"][:, :9]), ValueError), (bad(C=k["C"][..., :8]), ValueError), (bad(D=k["D"][:5]), ValueError),
                 (bad(h0=k["h0"][:1]), ValueError), (bad(x=k["x"].cpu()), TypeError), (bad(z=k["z"][:, ::2]), ValueError),
                 (lambda: gdn.scan_forward(**k, cu_seqlens=cu), ValueError),
                 (bad(B=k["B"].expand(2, 10, 3, 16), C=k["C"].expand(2, 10, 3, 16)), ValueError),
                 (lambda: gdn.scan_forward(k["x"], k["dt"], torch.zeros(32, 129, device=DEV), torch.zeros(2, 10, 129, device=DEV, dtype=BF),
                                           torch.zeros(2, 10, 129, device=DEV, dtype=BF)), gdn.GdnError),
                 (lambda: gdn.scan_backward(**k, dy=dy), ValueError),
                 (lambda: gdn.scan_backward(**k, dy=dy, saved=saved[:16]), gdn.GdnError),
                 (lambda: gdn.scan_step(k["x"], k["dt"], k["A"], k["B"], k["C"]), ValueError)):
        with pytest.raises(e):
            f()
