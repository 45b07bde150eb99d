"""GPU tests of the gated linear recurrence over many steps of its blocks: at least three each way in every layout (blocks alone with tiles of
64, 32 and 16 channels, clusters of 2, 4 and 8), so that the inputs' places, the exchange's and the barriers' phases are used again, and
a state or a gradient goes from step to step all the way.  dense and packed, rows that come by TMA and rows that do not.

Bounds, relative Frobenius per tensor, as in test_recur_gpu.py, with decays up to 0.999: a rounding of each of the 1000 decays that
count, 2^-25 each, all in one direction, is 3e-5; bf16 results are rounded once more, 2^-9."""
import pytest
import torch

import layers_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
TOL = {F32: 3e-5, BF: 2.0 ** -9 + 3e-5}
NAMES = ("dx", "drg", "dig", "dlam", "drg_bias", "dig_bias", "dz", "dh0")


@pytest.fixture()
def gdn():
    import __graft_entry__
    __graft_entry__.build()
    import chunkwise_delta_rule_02_gb300 as g
    return g


def layout(B, T, D, dtype, bwd, sms):
    """Runs a warp, blocks a cluster, steps of a block, as the library deals them (an odd width's forward has fewer warps, so more steps)."""
    W = (6 if dtype is BF else 4) if bwd else (12 if dtype is BF else 6)
    tiles = lambda q: B * -(-D // (64 // q))  # noqa: E731
    q = n = 1
    while q < 4 and tiles(2 * q) <= 2 * sms and 8 * W * q < T:
        q *= 2
    while q == 4 and n < 8 and tiles(4) * n * 2 <= 2 * sms and n * 8 * W * 4 < T:
        n *= 2
    return q, n, -(-T // (8 * W * q * n))


def dense(x, rg, ig, lam, rg_bias, ig_bias, z, h0):
    """The recurrence in the arguments' type: rows of one length, token by token."""
    r, i = torch.sigmoid(rg + rg_bias), torch.sigmoid(ig + ig_bias)
    m = 8.0 * torch.nn.functional.softplus(lam) * r
    a, u = torch.exp(-m), torch.sqrt(-torch.expm1(-2 * m)) * i * x
    h, rows = h0, []
    for at, ut in zip(a.unbind(1), u.unbind(1)):
        h = at * h + ut
        rows.append(h)
    return torch.stack(rows, 1) * z * torch.sigmoid(z), h


def plain(args, lens):
    if lens is None:
        return dense(*args)
    x, rg, ig, lam, rg_bias, ig_bias, z, h0 = args
    ys, ends, lo = [], [], 0
    for n, length in enumerate(lens):
        hi = lo + length
        y, h = dense(x[:, lo:hi], rg[:, lo:hi], ig[:, lo:hi], lam, rg_bias, ig_bias, z[:, lo:hi], h0[n:n + 1]) if length else (None, h0[n:n + 1])
        ys += [] if y is None else [y]
        ends.append(h)
        lo = hi
    return torch.cat(ys, 1), torch.cat(ends)


#: B, T, D, type, lengths, runs a warp and blocks a cluster forward (on 152 SMs)
CASES = [
    (40, 700, 256, BF, None, 1, 1), (8, 700, 1000, BF, None, 2, 1), (4, 1300, 1000, BF, None, 4, 1), (2, 2500, 1000, BF, None, 4, 2),
    (1, 5000, 1000, BF, None, 4, 4), (1, 9300, 64, BF, None, 4, 8),
    (8, 700, 1001, BF, None, 2, 1), (1, 5000, 1001, BF, None, 4, 4), (1, 9300, 63, BF, None, 4, 8),
    (40, 350, 256, F32, None, 1, 1), (4, 700, 1000, F32, None, 4, 1), (1, 4700, 40, F32, None, 4, 8),
    (2, 1300, 1001, F32, None, 4, 2), (1, 4700, 39, F32, None, 4, 8),
    (1, 9300, 64, BF, [3000, 0, 1, 6200, 99], 4, 8), (1, 5000, 1000, BF, [1537, 2, 3000, 0, 461], 4, 4), (1, 700, 8000, BF, [1, 500, 199], 2, 1),
    (1, 4700, 40, F32, [4000, 300, 0, 400], 4, 8), (1, 4700, 39, F32, [100] * 47, 4, 8), (1, 900, 2500, F32, [1, 0, 880, 19], 4, 1),
]


@pytest.mark.parametrize("c", CASES, ids=["%dx%dx%d-%s-%s" % (c[0], c[1], c[2], str(c[3])[6:], "packed" if c[4] else "dense") for c in CASES])
def test_many_steps(gdn, c):
    B, T, D, dt, lens, runs, blocks = c
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms == 152:
        assert layout(B, T, D, dt, False, sms)[:2] == (runs, blocks)
        assert min(layout(B, T, D, dt, bwd, sms)[2] for bwd in (False, True)) >= 3
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s, k=F32, scale=1.0: (torch.randn(*s, generator=g) * scale).to(k).to(DEV)  # noqa: E731
    n = B if lens is None else len(lens)
    cu = None if lens is None else torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)
    m = -torch.log(0.5 + 0.499 * torch.rand(D, generator=g)) / 8
    lam = torch.log(torch.expm1(m)).to(DEV)
    args = [rnd(B, T, D, k=dt), rnd(B, T, D, k=dt), rnd(B, T, D, k=dt), lam, rnd(D, scale=0.3), rnd(D), rnd(B, T, D, k=dt), rnd(n, D)]
    dy, dhT = rnd(B, T, D, k=dt), rnd(n, D)
    y, hT, saved = gdn.recur_forward(*args, cu_seqlens=cu, save=True)
    got = gdn.recur_backward(*args, dy=dy, dhT=dhT, saved=saved, cu_seqlens=cu)
    leaves = [t.double().requires_grad_() for t in args]
    ry, rh = plain(leaves, lens)
    ((ry * dy.double()).sum() + (rh * dhT.double()).sum()).backward()
    off = {"y": ref.err(y, ry.detach().cpu()), "hT": ref.err(hT, rh.detach().cpu())}
    off.update({k: ref.err(got[k], t.grad.cpu()) for k, t in zip(NAMES, leaves)})
    tol = {k: TOL[{"y": y, "hT": hT, **got}[k].dtype] for k in off}
    assert all(off[k] <= tol[k] for k in off), {k: v for k, v in off.items() if v > tol[k]}
