"""GPU tests of the linear softmax cross entropy against its definition in 64 bits: types, sizes from one token, feature and
entry to several tiles and pieces of the vocabulary, strides, ignored and bad targets, large logits, gradients (against the formula's
and against differences), streams and graphs, refusals.

Bounds.  loss, lse: a logit is a float32 sum of K products that are exact (bf16) or 2^-22 off (float32 in planes); the sum is off by at
most K 2^-24 of the terms' size, a random walk of sqrt(K) 2^-24 in fact, and the exponent by 2^-23 of it: 1e-5 (1 + |lse|) has a margin of several.
Gradients, relative Frobenius: bf16 rounds D once and the result once, 2^-9 / 1.15 each as rms, 2^-8 in all at most; float32 1e-5. To either
comes what logits of a size bring: lse and the logit are float32 numbers, each half a step of 2^-24 of its size off, and the sums
that gave them as much again, so that a probability is 4 max |lse| 2^-24 of itself off."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 1e-5, BF: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture()
def gdn():
    import chunkwise_delta_rule_02_gb300 as g
    return g


def plain(x, w, t, dloss=None, ignore=-100):
    """loss, lse (and dx, dw) in 64 bits."""
    K = x.shape[-1]
    x2, w2, t2 = x.double().reshape(-1, K), w.double(), t.reshape(-1)
    logits = x2 @ w2.t()
    lse = torch.logsumexp(logits, 1)
    some = (t2 >= 0) & (t2 < w.shape[0]) & (t2 != ignore)
    at = torch.where(some, t2, 0)
    loss = torch.where(some, lse - logits.gather(1, at[:, None])[:, 0], 0.0)
    if dloss is None:
        return loss.view(t.shape), lse.view(t.shape)
    d = torch.exp(logits - lse[:, None])
    d[torch.arange(len(at), device=DEV), at] -= 1
    d *= torch.where(some, dloss.double().reshape(-1), 0.0)[:, None]
    return loss.view(t.shape), lse.view(t.shape), (d @ w2).view(x.shape), d.t() @ x2


def err(got, want):
    n = float(want.norm())
    e = float((got.double() - want).norm())
    return e / n if n else e


def make(shape, V, dtype, seed=1, scale=2.0, ignored=0.1):
    g = torch.Generator().manual_seed(seed)
    K = shape[-1]
    x = torch.randn(*shape, generator=g).to(dtype).to(DEV)
    w = (torch.randn(V, K, generator=g) * scale * K ** -0.5).to(dtype).to(DEV)
    t = torch.randint(0, V, shape[:-1], generator=g)
    t[torch.rand(shape[:-1], generator=g) < ignored] = -100
    return x, w, t.to(DEV), torch.randn(shape[:-1], generator=g).to(DEV)


def check(gdn, x, w, t, dloss):
    loss, lse = gdn.xent_forward(x, w, t)
    g = gdn.xent_backward(x, w, t, lse, dloss)
    rl, rs, rx, rw = plain(x, w, t, dloss)
    room = 1e-5 * (1 + rs.abs())
    assert bool(((lse - rs).abs() <= room).all()) and bool(((loss - rl).abs() <= 2 * room).all())
    for n, want in (("dx", rx), ("dw", rw)):
        assert g[n].dtype == x.dtype and g[n].shape == want.shape
        e = err(g[n], want)
        assert e <= TOL[x.dtype] + 4 * float(rs.abs().max()) * 2.0 ** -24, (n, e)
    return loss, lse, g


SHAPES = [((1, 1), 1), ((1, 64), 5), ((3, 8), 300), ((7, 40), 257), ((128, 64), 256), ((129, 72), 512), ((257, 128), 1000), ((2, 100, 203), 777),
          ((300, 1), 2), ((5, 515), 40), ((32, 64), 3000), ((33, 48), 20000), ((64, 24), 40001), ((65, 136), 700), ((128, 200), 25000), ((1, 256), 50000), ((600, 320), 1300), ((4, 1, 16), 30), ((1, 9, 24), 70)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape,V", SHAPES)
def test_values_and_gradients(gdn, shape, V, dtype):
    check(gdn, *make(shape, V, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [24, 21, 20, 36, 75])
def test_pieces_of_the_vocabulary(gdn, dtype, K):
    """Tokens enough that the logits' gradients go by several pieces, the last one odd; row tiles of more than one group; widths that
    are a multiple of 8, of 4 and of nothing, with the sums of dx over pieces."""
    check(gdn, *make((70001, K), 3001 if dtype is BF else 1111, dtype))


@pytest.mark.parametrize("M", [3, 50, 300])
@pytest.mark.parametrize("K", [21, 4, 76])
def test_rows_that_end_within_16_bytes(gdn, M, K):
    """Aligned rows of a width that is no multiple of 8 in a buffer of NaN: what lies behind a row is not read."""
    x, w, t, dloss = make((M, K), 500, BF, 17)
    wide = (K + 15) // 8 * 8
    bx, bw = (torch.full((n, wide), float("nan"), dtype=BF, device=DEV) for n in (M, 500))
    bx[:, :K], bw[:, :K] = x, w
    check(gdn, bx[:, :K], bw[:, :K], t, dloss)


@pytest.mark.parametrize("T,B", [(7, 10001), (70001, 1)])
def test_pieces_into_rows_of_other_strides(gdn, T, B):
    """The library call with a dx whose rows lie apart: the same gradients, and nothing between them is touched."""
    from chunkwise_delta_rule_02_gb300 import layers
    for K in (24, 21):
        x, w, t, dloss = make((B, T, K), 2500, BF, 16)
        _, lse = gdn.xent_forward(x, w, t)
        want = gdn.xent_backward(x, w, t, lse, dloss)
        big = torch.full((B, T + 2, K + 11), 7.0, dtype=BF, device=DEV)
        dx, dw = big[:, 1:T + 1, 8:K + 8], torch.empty_like(w)
        shape = layers.xent_shape(x, w)
        ws = torch.empty(layers.dn_xent_workspace_size(shape, x, w, True), dtype=torch.uint8, device=DEV)
        layers.dn_xent_bwd(shape, x, w, t, lse, dloss, dx, dw, ws)
        assert torch.equal(dx, want["dx"]) and torch.equal(dw, want["dw"])
        big[:, 1:T + 1, 8:K + 8] = 7.0
        assert bool((big == 7.0).all())


def test_many_tiles_a_pair(gdn):
    check(gdn, *make((5000, 256), 9000, BF))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_views(gdn, dtype):
    """Slices of wider arrays (aligned and not), a sequence without its last token, targets one on, one gradient for all tokens."""
    x, w, t, dloss = make((3, 40, 64), 90, dtype, 3)
    want = check(gdn, x, w, t, dloss)

    def same(x2, w2, t2, d2):
        loss, lse = gdn.xent_forward(x2, w2, t2)
        g = gdn.xent_backward(x2, w2, t2, lse, d2)
        assert torch.equal(loss, want[0]) and torch.equal(lse, want[1]) and torch.equal(g["dx"], want[2]["dx"]) and torch.equal(g["dw"], want[2]["dw"])

    for pad in (8, 3):
        big = torch.full((4, 50, 64 + 2 * pad), float("nan"), dtype=dtype, device=DEV)
        bigw = torch.full((90, 64 + 2 * pad), float("nan"), dtype=dtype, device=DEV)
        xs, ws = big[1:, 5:45, pad:64 + pad], bigw[:, pad:64 + pad]
        xs.copy_(x)
        ws.copy_(w)
        wide = torch.zeros(3, 41, dtype=torch.int64, device=DEV)
        wide[:, 1:] = t
        same(xs, ws, wide[:, 1:], dloss.t().contiguous().t())
    turned = x.transpose(0, 1).contiguous().transpose(0, 1)
    same(turned, w, t, dloss)
    one = torch.full((), 0.25, device=DEV).expand(3, 40)
    _, lse = gdn.xent_forward(x, w, t)
    a, b = gdn.xent_backward(x, w, t, lse, one), gdn.xent_backward(x, w, t, lse, one.contiguous())
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"])
    row = x[:1, :1].expand(3, 40, 64)
    check(gdn, row, w, t, dloss)


def test_all_ignored_and_none(gdn):
    x, w, t, dloss = make((300, 32), 500, BF, 4)
    t[:] = -100
    loss, lse = gdn.xent_forward(x, w, t)
    g = gdn.xent_backward(x, w, t, lse, dloss)
    assert not bool(loss.any()) and not bool(g["dx"].any()) and not bool(g["dw"].any())
    assert bool(((lse - plain(x, w, t)[1]).abs() < 1e-4).all())
    for shape in ((0, 32), (0, 5, 32), (3, 0, 32)):
        e = x.new_empty(shape)
        te = t.new_empty(shape[:-1])
        loss, lse = gdn.xent_forward(e, w, te)
        g = gdn.xent_backward(e, w, te, lse, torch.empty(shape[:-1], device=DEV))
        assert loss.shape == shape[:-1] and g["dx"].shape == shape and not bool(g["dw"].any())


def test_ignore_index_of_the_caller(gdn):
    x, w, t, dloss = make((50, 16), 20, F32, 5, ignored=0.0)
    loss, lse = gdn.xent_forward(x, w, t, ignore_index=7)
    g = gdn.xent_backward(x, w, t, lse, dloss, ignore_index=7)
    rl, _, rx, rw = plain(x, w, t, dloss, ignore=7)
    assert bool((t == 7).any()) and float((loss - rl).abs().max()) < 1e-4 and err(g["dx"], rx) < 1e-5 and err(g["dw"], rw) < 1e-5


@pytest.mark.parametrize("bad", [-1, 90, 1 << 40])
def test_targets_outside_the_vocabulary(gdn, bad):
    x, w, t, dloss = make((40, 64), 90, BF, 6)
    good = t.clone()
    good[11] = -100
    want = gdn.xent_forward(x, w, good)
    wg = gdn.xent_backward(x, w, good, want[1], dloss)
    t[11] = bad
    with pytest.raises(gdn.GdnError):
        gdn.xent_forward(x, w, t)
    with pytest.raises(gdn.GdnError):
        gdn.xent_backward(x, w, t, want[1], dloss)
    loss, lse = gdn.xent_forward(x, w, t, check_status=False)
    g = gdn.xent_backward(x, w, t, lse, dloss, check_status=False)
    assert torch.equal(loss, want[0]) and torch.equal(g["dx"], wg["dx"]) and torch.equal(g["dw"], wg["dw"])


def test_large_logits(gdn):
    """Logits of some thousands: the maximum is taken out; probabilities of 0 and 1, losses of thousands."""
    x, w, t, dloss = make((200, 64), 700, F32, 7, scale=1000.0)
    check(gdn, x, w, t, dloss)
    x, w, t, dloss = make((200, 64), 700, BF, 8, scale=1000.0)
    check(gdn, x, w, t, dloss)
    low = -x.abs() - 1                       # all logits far below 0
    check(gdn, low, w.abs() + 1, t, dloss)


@pytest.mark.parametrize("M", [40, 300])
def test_losses_of_many_features(gdn, M):
    """The sums of 9001 products are rounded, not cut off: a cut is a step of 2^-24 of the sum down each of 560 times, 1.7e-5 of the logit's own
    size in the same direction, of which sums in segments of 1024 leave 64 steps a segment, 4e-6."""
    x, w, t, _ = make((M, 9001), 200, BF, 20, ignored=0.0)
    _, lse = gdn.xent_forward(x, w, t)
    _, want = plain(x, w, t)
    assert abs(float((lse.double() - want).mean())) <= 4e-6 * float((1 + want.abs()).mean())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_logits_far_below_zero(gdn, dtype):
    """All logits near -400, an odd vocabulary: exp(-lse) is infinite, and nothing of it reaches a gradient.

    The entries' common feature cancels in dx (the gradients of a token's logits sum to 0), their roundings do not, so what dx and dw may be
    off is counted from the terms: D of a bf16 call is off by half a step 2^-8 of itself, of a float32 call by 2^-22; the probability by
    4 |lse| 2^-24; the sums by their number of terms times 2^-24; and the result is rounded once."""
    x, w, t, dloss = make((300, 64), 501, dtype, 18, scale=0.5)
    x[:, 0], w[:, 0] = 20.0, -20.0
    loss, lse = gdn.xent_forward(x, w, t)
    g = gdn.xent_backward(x, w, t, lse, dloss)
    rl, rs, rx, rw = plain(x, w, t, dloss)
    room = 1e-5 * (1 + rs.abs())
    assert bool(((lse - rs).abs() <= room).all()) and bool(((loss - rl).abs() <= 2 * room).all())
    terms = torch.exp(x.double() @ w.double().t() - rs[:, None])
    terms[torch.arange(300, device=DEV), t.clamp(min=0)] += 1
    terms *= torch.where(t >= 0, dloss.double().abs(), 0.0)[:, None]
    off = (2.0 ** -8 if dtype is BF else 2.0 ** -22) + (4 * float(rs.abs().max()) + 501) * 2.0 ** -24
    for n, want, size in (("dx", rx, terms @ w.double().abs()), ("dw", rw, terms.t() @ x.double().abs())):
        assert bool(((g[n].double() - want).abs() <= off * size + (2.0 ** -8 if dtype is BF else 2.0 ** -24) * want.abs()).all()), n


def test_infinities_and_nan_stay_in_their_rows(gdn):
    """A token whose hidden state is not finite has no finite loss; the others' losses and dx are what they are without it."""
    x, w, t, dloss = make((300, 64), 400, BF, 9, ignored=0.0)
    loss, lse = gdn.xent_forward(x, w, t)
    g = gdn.xent_backward(x, w, t, lse, dloss)
    x[17, 3], x[200, 60] = float("nan"), float("inf")
    loss2, lse2 = gdn.xent_forward(x, w, t)
    g2 = gdn.xent_backward(x, w, t, lse2, dloss)
    rest = torch.ones(300, dtype=torch.bool, device=DEV)
    rest[17] = rest[200] = False
    assert torch.equal(loss[rest], loss2[rest]) and torch.equal(g["dx"][rest], g2["dx"][rest])
    assert not bool(torch.isfinite(loss2[~rest]).any())


@pytest.mark.parametrize("dtype,M,K", [(BF, 3, 16), (BF, 12, 21), (BF, 300, 64), (BF, 300, 37), (BF, 70001, 8), (F32, 11, 20), (F32, 300, 37)])
def test_padding_tokens_reach_nothing(gdn, dtype, M, K):
    """Hidden states, dloss and lse of tokens without a target hold NaN and infinities: losses and gradients to the bit as with zeros there."""
    x, w, t, dloss = make((M, K), 400, dtype, 19, ignored=0.4)
    t[1], t[2] = -100, 5
    pad = t < 0
    x[pad] = 0
    loss, lse = gdn.xent_forward(x, w, t)
    want = gdn.xent_backward(x, w, t, lse, dloss)
    x[pad] = float("nan")
    x[1] = float("inf")
    dloss[pad] = float("nan")
    loss2, lse2 = gdn.xent_forward(x, w, t)
    assert torch.equal(loss, loss2) and not bool(loss2[pad].any()) and torch.equal(lse[~pad], lse2[~pad])
    lse2[pad] = float("-inf")
    g = gdn.xent_backward(x, w, t, lse2, dloss)
    assert torch.equal(g["dx"], want["dx"]) and torch.equal(g["dw"], want["dw"]) and not bool(g["dx"][pad].any())


def test_gradients_against_differences(gdn):
    """Central differences along random directions, float32: the step 2^-5 leaves some 1e-3 of the derivative, the losses' rounding 1e-4."""
    x, w, t, dloss = make((60, 48), 130, F32, 10)
    _, lse = gdn.xent_forward(x, w, t)
    g = gdn.xent_backward(x, w, t, lse, dloss)
    gen = torch.Generator().manual_seed(11)
    for n in ("x", "w"):
        d = torch.randn((x if n == "x" else w).shape, generator=gen).to(DEV)
        v = [float((gdn.xent_forward(x + e * d if n == "x" else x, w + e * d if n == "w" else w, t)[0].double() * dloss).sum())
             for e in (2.0 ** -5, -2.0 ** -5)]
        along, size = float((g["d" + n].double() * d).sum()), float(g["d" + n].double().norm())
        assert abs((v[0] - v[1]) * 16 - along) <= 2e-2 * size


def test_runs_repeat_to_the_bit(gdn):
    x, w, t, dloss = make((900, 200), 2500, BF, 12)
    first = None
    for _ in range(3):
        loss, lse = gdn.xent_forward(x, w, t)
        g = gdn.xent_backward(x, w, t, lse, dloss)
        now = (loss, lse, g["dx"], g["dw"])
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_in_a_graph_and_on_two_streams(gdn):
    """Captured once and replayed on new inputs; two calls at once on streams of their own: the bits of the plain calls."""
    a, b = make((400, 128), 900, BF, 13), make((400, 128), 900, BF, 14)

    def both(x, w, t, dloss):
        loss, lse = gdn.xent_forward(x, w, t, check_status=False)
        g = gdn.xent_backward(x, w, t, lse, dloss, check_status=False)
        return loss, lse, g["dx"], g["dw"]

    want = both(*a), both(*b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(3):
        for i, (st, k) in enumerate(zip(streams, (a, b))):
            with torch.cuda.stream(st):
                got[i].append(both(*k))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(p, q) for o in got[i] for p, q in zip(o, want[i]))
    graph = torch.cuda.CUDAGraph()
    slot = [v.clone() for v in a]
    with torch.cuda.graph(graph):
        out = both(*slot)
    for k, w_ in ((a, want[0]), (b, want[1])):
        for s, v in zip(slot, k):
            s.copy_(v)
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(out, w_))


def test_refusals(gdn):
    x, w, t, dloss = make((20, 16), 30, BF, 15)
    _, lse = gdn.xent_forward(x, w, t)
    for args in ((x[0], w, t), (x, w[:, :8], t), (x, w, t[:5]), (x, w[0], t), (x[:, ::2], w[:, ::2].contiguous(), t), (x, w[:0], t)):
        with pytest.raises(ValueError):
            gdn.xent_forward(*args)
    for args in ((x, w.float(), t), (x, w, t.int()), (x.half(), w.half(), t), (x, w, t.cpu()), (x, w.cpu(), t)):
        with pytest.raises(TypeError):
            gdn.xent_forward(*args)
    with pytest.raises(TypeError):
        gdn.xent_backward(x, w, t, lse, dloss.bfloat16())
    with pytest.raises(ValueError):
        gdn.xent_backward(x, w, t, lse[:5], dloss)
    with pytest.raises(ValueError):
        gdn.xent_backward(x, w, t, lse, dloss[:5])
    small = torch.zeros(256, dtype=torch.uint8, device=DEV)
    with pytest.raises(gdn.GdnError):
        gdn.xent_forward(x, w, t, ws=small)
    with pytest.raises(gdn.GdnError):
        gdn.xent_backward(x, w, t, lse, dloss, ws=small)
