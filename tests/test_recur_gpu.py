"""GPU tests of the gated linear recurrence against its plain 64-bit form: types, odd widths, lengths from none to
several steps of a cluster's blocks, strides, packed sequences with empty and one-token members, extreme gates, infinities
and NaN, single tokens, a captured training step; gradients against the formula's (by differentiation) and against differences.

Bounds, relative Frobenius per tensor.  A bf16 result is a float32 one rounded once: 2^-9 (half a step of 2^-8, spread
over significands, is 1.7e-3).  float32 results: the gates, the decay and the square root are off by a few 2^-22 (an ex2, a reciprocal and an rsqrt
of 2^-22 each, their arguments' roundings), so a state, whose error is that of each input's weight
exp(-sum m) with sum m of order 1 where the weight counts, by about 2^-20; 1e-5 leaves a factor of ten for sums over the tokens."""
import pytest
import torch

import layers_ref as ref
import recur_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 1e-5, BF: 2.0 ** -9 + 1e-5}
GRADS = ("dx", "drg", "dig", "dlam", "drg_bias", "dig_bias", "dz", "dh0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture()
def gdn():
    import chunkwise_delta_rule_02_gb300 as g
    return g


def close(got, want, dtype=None):
    e = ref.err(got, want)
    assert e <= TOL[dtype or got.dtype], e


CASES = [  # B, T, D, dtype, bias, gate, state, lengths
    (2, 70, 64, BF, True, True, True, None),
    (1, 1, 2, F32, False, False, False, None),
    (3, 7, 1, F32, True, True, True, None),
    (2, 8, 130, BF, True, False, False, None),
    (1, 9, 501, F32, True, False, True, None),
    (2, 65, 129, BF, False, True, True, None),             # odd width: one element an access
    (1, 1100, 70, F32, True, True, False, None),           # several steps of eight blocks
    (1, 515, 64, BF, True, False, True, None),             # one step and a token run
    (40, 130, 256, BF, True, True, False, None),           # rows enough for blocks without a cluster
    (2, 0, 16, F32, True, True, True, None),               # no tokens
    (1, 140, 66, BF, True, True, True, [0, 1, 70, 0, 2, 64, 3, 0]),
    (1, 131, 37, F32, True, False, False, [64, 1, 66]),
    (1, 700, 128, F32, False, True, True, [1, 511, 1, 187]),
    (1, 24, 8, BF, True, False, True, [1] * 24),
    (1, 0, 8, BF, True, False, True, [0, 0]),
    # channels enough for tiles of 64, in clusters and alone, by boxes, words and elements
    (5, 300, 640, BF, True, True, True, None),
    (3, 200, 1000, F32, True, True, True, None),
    (2, 330, 1302, BF, True, True, True, None),
    (2, 330, 1301, BF, True, False, True, None),
    (2, 130, 1301, F32, True, True, False, None),
    (1, 700, 1304, BF, True, True, True, [0, 100, 1, 300, 299, 0]),
    (1, 600, 1301, BF, True, True, True, [599, 1]),
    (1, 300, 1301, F32, False, True, True, [1, 2, 3, 294]),
    (1, 2100, 24, BF, True, True, True, [700, 1400]),
]


def case(c, seed=1):
    B, T, D, dt, bias, gate, state, lens = c
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, dtype=F32, scale=1.0: (torch.randn(*s, generator=g) * scale).to(dtype).to(DEV)  # noqa: E731
    n = B if lens is None else len(lens)
    cu = None if lens is None else torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)
    lam = torch.log(torch.expm1(-torch.log(0.5 + 0.4999 * torch.rand(D, generator=g)) / 8)).to(DEV)     # decays of 0.5 to 0.9999
    return dict(args=(rnd(B, T, D, dtype=dt), rnd(B, T, D, dtype=dt), rnd(B, T, D, dtype=dt), lam),
                more=dict(rg_bias=rnd(D) if bias else None, ig_bias=rnd(D) if bias else None,
                          z=rnd(B, T, D, dtype=dt) if gate else None, h0=rnd(n, D) if state else None),
                cu=cu, dy=rnd(B, T, D, dtype=dt), dhT=rnd(n, D))


def want_of(k, dhT=True, grad=True):
    """(y, hT, gradients) in 64 bits."""
    leaves = [ref.d64(t) for t in k["args"]] + [ref.d64(t) for t in k["more"].values()]
    if grad:
        leaves = [None if t is None else t.clone().requires_grad_() for t in leaves]
    y, hT = recur_ref.recur(*leaves, cu=k["cu"])
    if not grad:
        return y, hT
    loss = (y * ref.d64(k["dy"])).sum()
    if dhT:
        loss = loss + (hT * ref.d64(k["dhT"])).sum()
    if loss.requires_grad:
        loss.backward()
    got = [None if t is None else (torch.zeros_like(t) if t.grad is None else t.grad) for t in leaves]
    names = ("dx", "drg", "dig", "dlam", "drg_bias", "dig_bias", "dz", "dh0")
    return y.detach(), hT.detach(), dict(zip(names, got))


@pytest.mark.parametrize("c", CASES)
def test_forward(gdn, c):
    k = case(c)
    y, hT = gdn.recur_forward(*k["args"], **k["more"], cu_seqlens=k["cu"])
    ry, rh = want_of(k, grad=False)
    close(y, ry)
    close(hT, rh)
    y2, none = gdn.recur_forward(*k["args"], **k["more"], cu_seqlens=k["cu"], want_state=False)
    assert none is None and torch.equal(y, y2)


@pytest.mark.parametrize("c", CASES)
@pytest.mark.parametrize("upstream_state", [False, True])
def test_backward(gdn, c, upstream_state):
    k = case(c, 2)
    _, _, saved = gdn.recur_forward(*k["args"], **k["more"], cu_seqlens=k["cu"], save=True)
    g = gdn.recur_backward(*k["args"], **k["more"], dy=k["dy"], dhT=k["dhT"] if upstream_state else None, saved=saved, cu_seqlens=k["cu"])
    _, _, want = want_of(k, dhT=upstream_state)
    for n in GRADS:
        assert (g[n] is None) == (want[n] is None), n
        if g[n] is not None:
            e = ref.err(g[n], want[n])
            assert e <= TOL[g[n].dtype], (n, e)


def inside(t, pad=2):
    """The same values as a strided view into a larger buffer of NaN: what lies around must not be read."""
    big = torch.full([n + 2 * pad for n in t.shape[:-1]] + [t.shape[-1] + 9], float("nan"), dtype=t.dtype, device=t.device)
    v = big[tuple(slice(pad, pad + n) for n in t.shape[:-1]) + (slice(5, 5 + t.shape[-1]),)]
    v.copy_(t)
    return v


@pytest.mark.parametrize("c", [CASES[0], CASES[6], CASES[10]])
def test_views_give_the_same(gdn, c):
    """Slices (unaligned), time-major arrays and a result written in place of a slice: the dense call's bits."""
    k = case(c, 3)
    kw = dict(k["more"], cu_seqlens=k["cu"])
    y, hT, saved = gdn.recur_forward(*k["args"], **kw, save=True)
    g = gdn.recur_backward(*k["args"], **kw, dy=k["dy"], dhT=k["dhT"], saved=saved)
    for f in (inside, lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)):
        x, rg, ig = (f(t) for t in k["args"][:3])
        kw2 = dict(kw, z=None if kw["z"] is None else f(kw["z"]))
        y2, hT2, saved2 = gdn.recur_forward(x, rg, ig, k["args"][3], **kw2, save=True, out=f(torch.zeros_like(y)))
        assert torch.equal(y, y2) and torch.equal(hT, hT2)
        g2 = gdn.recur_backward(x, rg, ig, k["args"][3], **kw2, dy=f(k["dy"]), dhT=k["dhT"], saved=saved2)
        for n in GRADS:
            assert g[n] is None and g2[n] is None or torch.equal(g[n], g2[n]), n


@pytest.mark.parametrize("dt,D", [(BF, 6), (BF, 70), (F32, 70), (F32, 66)])
def test_rows_that_end_within_16_bytes(gdn, dt, D):
    """Aligned rows of an even width in buffers of NaN: the dense call's values, and results leave what lies behind them."""
    k = case((2, 40, D, dt, True, True, True, None), 16)
    x, rg, ig, lam = k["args"]
    wide = (D + 15) // 8 * 8

    def aligned(t):
        big = torch.full(t.shape[:2] + (wide,), float("nan"), dtype=dt, device=DEV)
        big[..., :D] = t
        return big[..., :D]

    more = dict(k["more"], z=aligned(k["more"]["z"]))
    big = torch.full((2, 40, wide), 7.0, dtype=dt, device=DEV)
    y, hT, saved = gdn.recur_forward(aligned(x), aligned(rg), aligned(ig), lam, **more, out=big[..., :D], save=True)
    ry, rh, want = want_of(k)
    close(y, ry)
    close(hT, rh)
    assert bool((big[..., D:] == 7.0).all())
    g = gdn.recur_backward(aligned(x), aligned(rg), aligned(ig), lam, **more, dy=aligned(k["dy"]), dhT=k["dhT"], saved=saved)
    for n in GRADS:
        assert ref.err(g[n], want[n]) <= TOL[g[n].dtype], n


@pytest.mark.parametrize("dt,D", [(BF, 64), (BF, 9), (F32, 40), (F32, 10000)])
def test_many_short_sequences(gdn, dt, D):
    """More sequences than a warp holds, many of them within a warp's tokens, empty ones in rows, between long ones."""
    lens = [1] * 40 + [0] * 35 + [90] + [0, 0, 1, 2] * 12 + [20] * 3 + [0] * 33 + [130, 3] + [0] * 9 + [1] * 10
    k = case((1, sum(lens), D, dt, True, True, True, lens), 19)
    y, hT, saved = gdn.recur_forward(*k["args"], **k["more"], cu_seqlens=k["cu"], save=True)
    ry, rh, want = want_of(k)
    close(y, ry)
    close(hT, rh)
    g = gdn.recur_backward(*k["args"], **k["more"], dy=k["dy"], dhT=k["dhT"], saved=saved, cu_seqlens=k["cu"])
    for n in GRADS:
        assert ref.err(g[n], want[n]) <= TOL[g[n].dtype], n


@pytest.mark.parametrize("dt,D,pitch", [(BF, 37, 40), (BF, 67, 67), (BF, 130, 131), (F32, 37, 38), (F32, 67, 67), (F32, 130, 133)])
@pytest.mark.parametrize("B,T", [(2, 90), (40, 33)])
def test_rows_at_every_alignment(gdn, dt, D, pitch, B, T):
    """Each array starts at another offset from 16 bytes in a buffer of NaN that ends with it; odd distances of rows; few rows and many."""
    k = case((B, T, D, dt, True, True, True, None), 18)
    x, rg, ig, lam = k["args"]

    def at(t, o):
        big = torch.full((o + B * T * pitch - (pitch - D),), float("nan"), dtype=dt, device=DEV)
        v = big.as_strided((B, T, D), (T * pitch, pitch, 1), o)
        v.copy_(t)
        return v

    for o in range(0, 8 if dt is BF else 4, 3):
        a, more = (at(x, o), at(rg, o + 1), at(ig, o + 2), lam), dict(k["more"], z=at(k["more"]["z"], o + 5))
        y, hT, saved = gdn.recur_forward(*a, **more, save=True)
        ry, rh, want = want_of(k)
        close(y, ry)
        close(hT, rh)
        g = gdn.recur_backward(*a, **more, dy=at(k["dy"], o + 3), dhT=k["dhT"], saved=saved)
        for n in GRADS:
            assert ref.err(g[n], want[n]) <= TOL[g[n].dtype], n


def test_a_result_leaves_what_lies_around_it(gdn):
    k = case((2, 21, 35, BF, True, False, False, None), 4)
    big = torch.full((4, 30, 50), 7.0, dtype=BF, device=DEV)
    gdn.recur_forward(*k["args"], **k["more"], out=big[1:3, 4:25, 10:45])
    big[1:3, 4:25, 10:45] = 7.0
    assert bool((big == 7.0).all())


def test_gradients_against_differences(gdn):
    """Central differences of <y, dy> + <hT, dhT>, float32, along random directions: the step 2^-6 leaves an error of its
    square, some 1e-3 of the derivative, and of the sums' rounding, 1e-5."""
    k = case((2, 40, 34, F32, True, True, True, None), 5)
    names = ("x", "rg", "ig", "lam", "rg_bias", "ig_bias", "z", "h0")
    vals = dict(zip(names, list(k["args"]) + list(k["more"].values())))

    def loss(v):
        y, hT = gdn.recur_forward(*[v[n] for n in names[:4]], **{n: v[n] for n in names[4:]})
        return float((y.double() * k["dy"]).sum() + (hT.double() * k["dhT"]).sum())

    _, _, saved = gdn.recur_forward(*k["args"], **k["more"], save=True)
    g = gdn.recur_backward(*k["args"], **k["more"], dy=k["dy"], dhT=k["dhT"], saved=saved)
    gen = torch.Generator().manual_seed(6)
    for n in names:
        step = 2.0 ** -6
        d = torch.randn(vals[n].shape, generator=gen).to(DEV)
        up, down = (loss(dict(vals, **{n: vals[n] + e * d})) for e in (step, -step))
        along = float((g["d" + n if n not in ("rg_bias", "ig_bias") else "d" + n].double() * d).sum())
        size = float(g["d" + n].double().norm())
        assert abs((up - down) / (2 * step) - along) <= 2e-2 * size, n


@pytest.mark.parametrize("lam,rg", [(60.0, 0.0), (-60.0, 0.0), (-200.0, 0.0), (200.0, 3.0), (0.0, 60.0), (0.0, -60.0), (0.0, -200.0), (-5.0, float("-inf")),
                                    (-5.0, float("inf"))])
def test_extreme_gates(gdn, lam, rg):
    """A decay of 0 and one of 1: results and gradients are finite and the formula's (their limits, where 1 - a^2 is 0)."""
    T, D = 20, 4
    g = torch.Generator().manual_seed(7)
    x, ig, dy = (torch.randn(1, T, D, generator=g).to(DEV) for _ in range(3))
    rgs, lams = torch.full((1, T, D), rg, device=DEV), torch.full((D,), lam, device=DEV)
    h0 = torch.randn(1, D, generator=g).to(DEV)
    y, hT, saved = gdn.recur_forward(x, rgs, ig, lams, h0=h0, save=True)
    ry, _ = recur_ref.recur(*(ref.d64(t) for t in (x, rgs, ig, lams)), h0=ref.d64(h0))
    assert bool(torch.isfinite(y).all())
    # sqrt(1 - a^2) of an m that float32 cannot hold is 0 here, and below 1e-18 in 64 bits
    assert float((y.cpu().double() - ry).abs().max()) <= 1e-5 * (1 + float(ry.abs().max()))
    got = gdn.recur_backward(x, rgs, ig, lams, h0=h0, dy=dy, saved=saved)
    assert all(bool(torch.isfinite(v).all()) for v in got.values() if v is not None)
    if abs(lam) <= 60 and abs(rg) < 30:
        leaves = [ref.d64(t).clone().requires_grad_() for t in (x, rgs, ig, lams)]
        (recur_ref.recur(*leaves, h0=ref.d64(h0))[0] * ref.d64(dy)).sum().backward()
        for n, t in zip(("dx", "drg", "dig", "dlam"), leaves):
            assert float((got[n].cpu().double() - t.grad).abs().max()) <= 1e-4 * (1e-3 + float(t.grad.abs().max())), n


def test_infinities_and_nan_stay_in_their_sequence_and_channel(gdn):
    """A NaN and an infinity among the inputs reach what the recurrence carries them to and nothing else: as in 64 bits."""
    lens = [100, 1, 300, 0, 199]
    k = case((1, 600, 10, F32, True, False, True, lens), 8)
    x = k["args"][0]
    x[0, 120, 3], x[0, 40, 5], x[0, 450, 7] = float("nan"), float("inf"), float("-inf")
    y, hT = gdn.recur_forward(*k["args"], **k["more"], cu_seqlens=k["cu"])
    ry, rh = want_of(k, grad=False)
    for got, want in ((y.cpu().double(), ry), (hT.cpu().double(), rh)):
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want))
        fine = torch.isfinite(want)
        assert float((got - want)[fine].norm() / want[fine].norm()) <= 1e-5


def test_an_infinity_passes_decays_whose_product_underflows(gdn):
    """Over 600 tokens the product of decays of 0.5 is 0 in float32; an infinite state goes through each of them."""
    x = torch.zeros(1, 600, 3, device=DEV)
    lam = torch.full((3,), 1.0, device=DEV)
    h0 = torch.tensor([[float("inf"), 1.0, float("nan")]], device=DEV)
    y, hT = gdn.recur_forward(x, x, x, lam, h0=h0)
    assert bool(torch.isinf(y[..., 0]).all()) and bool(torch.isnan(y[..., 2]).all()) and bool(torch.isfinite(y[..., 1]).all())
    assert bool(torch.isinf(hT[0, 0])) and float(hT[0, 1]) == 0.0


@pytest.mark.parametrize("n,D,dt,gate", [(1, 1, F32, True), (5, 130, BF, True), (256, 64, BF, False), (3, 33, BF, True)])
def test_step(gdn, n, D, dt, gate):
    k = case((n, 1, D, dt, True, gate, True, None), 9)
    one = lambda t: None if t is None else t[:, 0]  # noqa: E731
    args, m = [one(t) for t in k["args"][:3]] + [k["args"][3]], k["more"]
    state = m["h0"].clone()
    y, new = gdn.recur_step(*args, rg_bias=m["rg_bias"], ig_bias=m["ig_bias"], z=one(m["z"]), state=state, out_state=state)
    ry, rh = want_of(k, grad=False)
    close(y, ry[:, 0])
    close(new, rh)
    assert new.data_ptr() == state.data_ptr()
    zero, _ = gdn.recur_step(*args, rg_bias=m["rg_bias"], ig_bias=m["ig_bias"], z=one(m["z"]))
    k["more"]["h0"] = None
    close(zero, want_of(k, grad=False)[0][:, 0])


def test_pieces_and_single_tokens_give_the_whole(gdn):
    """A prompt in two pieces and then token by token against the whole sequence: float32 states, so 1e-5."""
    k = case((2, 200, 66, F32, True, True, True, None), 10)
    whole, hT = gdn.recur_forward(*k["args"], **k["more"])
    m = k["more"]
    ys, h = [], m["h0"]
    for lo, hi in ((0, 77), (77, 150)):
        y, h = gdn.recur_forward(*[t[:, lo:hi] for t in k["args"][:3]], k["args"][3], **dict(m, z=m["z"][:, lo:hi], h0=h))
        ys.append(y)
    for t in range(150, 200):
        y, h = gdn.recur_step(*[v[:, t] for v in k["args"][:3]], k["args"][3], rg_bias=m["rg_bias"], ig_bias=m["ig_bias"], z=m["z"][:, t],
                              state=h, out_state=h)
        ys.append(y[:, None])
    close(torch.cat(ys, 1), whole.cpu().double())
    close(h, hT.cpu().double())


def test_malformed_offsets_raise(gdn):
    k = case(CASES[10], 11)
    for bad in ([0, 5, 3, 140], [0, 70, 141], [1, 140]):
        cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
        more = dict(k["more"], h0=None)
        with pytest.raises(gdn.GdnError):
            gdn.recur_forward(*k["args"], **more, cu_seqlens=cu)
        out = torch.full_like(k["dy"], 3.0)
        gdn.recur_forward(*k["args"], **more, cu_seqlens=cu, out=out, check_status=False)
        assert bool((out == 3.0).all())        # no sequence: no row is written


def test_runs_repeat_to_the_bit(gdn):
    k = case(CASES[6], 12)
    first = None
    for _ in range(3):
        y, hT, saved = gdn.recur_forward(*k["args"], **k["more"], save=True)
        g = gdn.recur_backward(*k["args"], **k["more"], dy=k["dy"], dhT=k["dhT"], saved=saved)
        now = [y, hT] + [v for v in g.values() if v is not None]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_training_step_in_a_graph_and_on_another_stream(gdn):
    """Forward and backward captured once, replayed on new inputs, and run on a side stream: the bits of the plain calls."""
    k = case(CASES[0], 13)
    k2 = case(CASES[0], 14)

    def both(k):
        y, hT, saved = gdn.recur_forward(*k["args"], **k["more"], save=True)
        g = gdn.recur_backward(*k["args"], **k["more"], dy=k["dy"], dhT=k["dhT"], saved=saved)
        return [y, hT] + [v for v in g.values() if v is not None]

    want, want2 = both(k), both(k2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = both(k)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, there))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(k)
    for a, b in zip(list(k["args"]) + list(k["more"].values()) + [k["dy"], k["dhT"]],
                    list(k2["args"]) + list(k2["more"].values()) + [k2["dy"], k2["dhT"]]):
        a.copy_(b)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want2, out))


def test_refusals(gdn):
    k = case(CASES[0], 15)
    x, rg, ig, lam = k["args"]
    for args in ((x[0], rg, ig, lam), (x, rg[:, :3], ig, lam), (x, rg, ig, lam[:3]), (x, rg, ig[..., :4], lam), (x[..., ::2], rg, ig, lam)):
        with pytest.raises(ValueError):
            gdn.recur_forward(*args)
    for args in ((x, rg.float(), ig, lam), (x, rg, ig, lam.double()), (x.half(), rg.half(), ig.half(), lam)):
        with pytest.raises(TypeError):
            gdn.recur_forward(*args)
    for c in (-1.0, float("nan"), float("inf")):
        with pytest.raises(gdn.GdnError):
            gdn.recur_forward(x, rg, ig, lam, c=c)
    with pytest.raises(ValueError):
        gdn.recur_forward(x, rg, ig, lam, h0=torch.zeros(3, 64, device=DEV))
    with pytest.raises(ValueError):
        gdn.recur_forward(x, rg, ig, lam, cu_seqlens=torch.tensor([0, 140], dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        gdn.recur_backward(x, rg, ig, lam)
    with pytest.raises(gdn.GdnError):
        gdn.recur_backward(x, rg, ig, lam, dy=k["dy"], saved=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(gdn.GdnError):
        gdn.recur_backward(x, rg, ig, lam, dy=k["dy"], saved=torch.zeros(1 << 16, dtype=torch.uint8, device=DEV), ws=torch.zeros(16, dtype=torch.uint8, device=DEV))
