"""GPU tests of the selective state space scan over several time segments: what is not finite stays in its
sequence and goes through the segments as through one recurrence; every layout of states over lanes, dense and
packed.  Bounds as in test_scan_gpu: the inputs are made alike, with memories of the same length."""
import pytest
import torch

import layers_ref as ref
from test_scan_gpu import BF, F32, TOL, close, make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture()
def gdn():
    import chunkwise_delta_rule_02_gb300 as g
    return g


def segmented(x, Bm):
    """Whether both passes over one row of few channels are cut into time segments: their workspaces then hold the
    segments' states (the backward's beside dB's and dC's partial results and one row of sums over tokens)."""
    from chunkwise_delta_rule_02_gb300 import layers
    shape = layers.scan_shape(x, Bm)
    T, D, G, N = x.shape[1], x.shape[2], Bm.shape[2], Bm.shape[3]
    Np = max(8, 1 << (N - 1).bit_length())
    CH = 64 if N <= 16 else 32 if N <= 32 else 8            # channels of a block
    tiles = G * -(-(D // G) // CH)
    uncut = 4 * (tiles * T * 2 * Np + D * Np + 2 * D) + 4 * 256
    return layers.dn_scan_workspace_size(shape) > 256 and layers.dn_scan_workspace_size(shape, True) > uncut


def inputs(T, D, N, lens=None, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(DEV)  # noqa: E731
    n = 1 if lens is None else len(lens)
    cu = None if lens is None else torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)
    # A to -16 and steps about 0.1: a segment's decay product is 0 in float32, a single token's is not
    k = dict(x=r(1, T, D), dt=r(1, T, D, scale=0.5), A=-torch.linspace(0.5, 16.0, N).repeat(D, 1).to(DEV), B=r(1, T, 1, N),
             C=r(1, T, 1, N), D=r(D), z=r(1, T, D), dt_bias=torch.full((D,), -2.2, device=DEV), h0=r(n, D, N, scale=0.5))
    return k, cu


@pytest.mark.parametrize("N", [16, 48])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_reaches_the_end_of_its_sequence(gdn, N, bad):
    T, D = 2000, 20
    k, _ = inputs(T, D, N)
    assert segmented(k["x"], k["B"])
    clean, hc = gdn.scan_forward(**k)
    k["x"][0, 100, 3] = bad
    y, hT = gdn.scan_forward(**k)
    v = {n: ref.d64(t) for n, t in k.items()}
    _, rh = ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"], v["h0"])
    rh = rh[0, 3]
    assert not torch.isfinite(rh).any()
    assert torch.equal(torch.isnan(hT[0, 3]).cpu(), torch.isnan(rh))
    assert torch.equal(torch.isposinf(hT[0, 3]).cpu(), torch.isposinf(rh))
    assert not torch.isfinite(y[0, 100:, 3]).any() and torch.equal(y[0, :100], clean[0, :100])
    rest = [c for c in range(D) if c != 3]
    assert torch.equal(y[..., rest], clean[..., rest]) and torch.equal(hT[:, rest], hc[:, rest])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_ends_at_a_sequence_start(gdn, bad):
    lens = [700, 0, 1, 799, 500]
    k, cu = inputs(2000, 20, 16, lens, 2)
    assert segmented(k["x"], k["B"])
    clean, hc = gdn.scan_forward(**k, cu_seqlens=cu)
    k["x"][0, 800, 3] = bad        # in the fourth sequence, tokens 701 .. 1499
    y, hT = gdn.scan_forward(**k, cu_seqlens=cu)
    assert not torch.isfinite(y[0, 800:1500, 3]).any() and not torch.isfinite(hT[3, 3]).any()
    assert torch.equal(y[0, 1500:], clean[0, 1500:]) and torch.equal(y[0, :800], clean[0, :800])
    others = [0, 1, 2, 4]
    assert torch.equal(hT[others], hc[others])


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_gradient_that_is_not_finite_reaches_the_start_of_its_sequence(gdn, packed, bad):
    k, cu = inputs(2000, 20, 16, [700, 0, 1, 799, 500] if packed else None, 3)
    assert segmented(k["x"], k["B"])
    g = torch.Generator().manual_seed(4)
    dy = torch.randn(1, 2000, 20, generator=g).to(DEV)
    _, _, saved = gdn.scan_forward(**k, cu_seqlens=cu, save=True)
    clean = gdn.scan_backward(**k, dy=dy, saved=saved, cu_seqlens=cu)
    dy[0, 1400, 3] = bad
    got = gdn.scan_backward(**k, dy=dy, saved=saved, cu_seqlens=cu)
    first, seq = (701, 3) if packed else (0, 0)
    for n in ("dx", "ddt"):
        assert not torch.isfinite(got[n][0, first:1401, 3]).any(), n
        assert torch.equal(got[n][0, :first], clean[n][0, :first]) and torch.equal(got[n][0, 1401:], clean[n][0, 1401:]), n
    assert not torch.isfinite(got["dh0"][seq, 3]).any()
    others = [s for s in range(k["h0"].shape[0]) if s != seq]
    assert torch.equal(got["dh0"][others], clean["dh0"][others])
    assert not torch.isfinite(got["dB"][0, first:1401]).any()
    assert torch.equal(got["dB"][0, :first], clean["dB"][0, :first]) and torch.equal(got["dB"][0, 1401:], clean["dB"][0, 1401:])


LAYOUTS = [  # D, N, G, dtype, T, lengths
    (100, 8, 1, F32, 400, None),
    (100, 8, 1, F32, 400, [150, 0, 1, 249]),
    (140, 16, 2, BF, 400, [63, 1, 0, 336]),
    (16, 32, 2, F32, 400, None),
    (80, 32, 2, F32, 400, [150, 0, 1, 249]),
    (70, 30, 1, BF, 400, [17, 383]),
    (20, 64, 1, F32, 300, None),
    (20, 64, 1, F32, 300, [150, 0, 1, 149]),
    (18, 33, 2, BF, 300, [0, 128, 172]),
    (12, 100, 1, F32, 300, None),
    (12, 100, 1, F32, 300, [150, 0, 1, 149]),
    (24, 128, 3, BF, 300, [1, 1, 298, 0]),
]


@pytest.mark.parametrize("c", LAYOUTS)
def test_every_layout_over_segments(gdn, c):
    """Forward and backward with initial states and gradients of the final ones."""
    D, N, G, dtype, T, lens = c
    k, cu, _, dy, dhT = make((1, T, D, N, G, dtype, True, True, True, True, True, lens), 5)
    assert segmented(k["x"], k["B"])
    y, hT, saved = gdn.scan_forward(**k, cu_seqlens=cu, save=True)
    g = gdn.scan_backward(**k, dy=dy, dhT=dhT, saved=saved, cu_seqlens=cu)
    v = {n: ref.leaf(t) for n, t in k.items()}
    outs = ref.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"], v["h0"], cu=cu)
    close(y, outs[0])
    close(hT, outs[1])
    want = dict(zip(k, ref.grads(outs, (ref.d64(dy), ref.d64(dhT)), list(v.values()))))
    for n in k:
        got = g["d" + n]
        # sums over tokens and channels of terms of both signs: what they cancel stays as error
        assert ref.err(got, want[n]) <= (4 if n in ("A", "dt_bias", "dt", "h0") and got.dtype == F32 else 1) * TOL[got.dtype], n
