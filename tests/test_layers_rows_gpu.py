"""GPU tests at sizes where a thread goes on to further rows or sequences: the norm's passes over many rows (a
group's next row within a (batch, head), past its end, and the sums of dw over many rows), and the single-token
scan with two sequences a lane, the last of them missing.

Bounds, relative Frobenius per tensor.  bf16 results: as in test_layers_gpu, one rounding to 8 significant bits is
2^-8 / sqrt(3) / 1.4 over many elements, 2^-9 is asked (norm), 2^-8 (scan).  float32 results: products of a few
factors good to 2^-22 each; sums over all rows of terms of both signs, taken in runs of at most 30 to 80 terms one
after another and then over the blocks: their roundings add up like the terms themselves, so that a sum is off by some
sqrt(80) 2^-24 = 5e-7 of itself: 5e-6 is asked.  The scan's single token: 4e-6, as in test_scan_gpu."""
import pytest
import torch

import layers_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
NORM_TOL = {F32: 5e-6, BF: 2.0 ** -9 + 5e-6}
SCAN_TOL = {F32: 4e-6, BF: 2.0 ** -8 + 4e-6}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture()
def gdn():
    import chunkwise_delta_rule_02_gb300 as g
    return g


NORM = [  # B, H, T, d, dtype, gate, residual, scale, per head
    (2, 3, 10007, 128, BF, True, False, False, False),      # 16 rows at a time, T not a multiple of them
    (2, 3, 10007, 128, BF, True, False, False, True),
    (5, 4, 3001, 100, F32, True, True, True, False),
    (1, 1, 61001, 256, BF, False, True, True, False),
    (30011, 2, 1, 128, BF, True, False, False, False),      # every next row in another (batch, head)
    (4001, 3, 5, 128, F32, False, False, False, True),      # T smaller than the rows taken at a time
    (2, 1, 2003, 2048, BF, False, True, True, False),       # a row a block
    (2, 1, 2003, 2048, BF, False, True, False, False),
    (1, 3, 1301, 129, F32, True, False, False, False),      # the same, one element an access
    (3, 1, 1500, 1025, BF, False, True, True, False),
]


@pytest.mark.parametrize("c", NORM)
def test_norm_over_many_rows(gdn, c):
    B, H, T, d, dt, gate, res, scaled, per = c
    gen = torch.Generator().manual_seed(1)
    r = lambda *s, dtype=F32, scale=1.0: (torch.randn(*s, generator=gen) * scale).to(dtype).to(DEV)  # noqa: E731
    s = (B, H, T, d)
    x, w, z = r(*s, dtype=dt), r(H, d) if per else r(d), r(B, T, H, d, dtype=dt).transpose(1, 2) if gate else None
    residual, scale = r(*s, dtype=dt, scale=2.0) if res else None, r(d) if scaled else None
    dy, dsum = r(B, T, H, d, dtype=dt).transpose(1, 2), r(*s, dtype=dt) if res else None

    def close(got, want, name):
        e = ref.err(got, want)
        assert e <= NORM_TOL[got.dtype], (name, e)

    got = gdn.norm_forward(x, w, z=z, residual=residual, res_scale=scale)
    y, total = (got, x) if residual is None else got
    want, rr = ref.norm(*(ref.d64(t) for t in (x, w, z, residual, scale)))
    close(y, want, "y")
    if res:
        close(total, rr, "sum")
    g = gdn.norm_backward(x, w, dy, z=z, sum=total if res else None, dsum=dsum, res_scale=scale)
    leaves = {n: ref.leaf(t) for n, t in (("r", total), ("w", w), ("z", z)) if t is not None}
    yy, _ = ref.norm(leaves["r"], leaves["w"], leaves.get("z"))
    grads = dict(zip(leaves, ref.grads((yy, leaves["r"]), (ref.d64(dy), ref.d64(dsum)), list(leaves.values()))))
    close(g["dx"], grads["r"] if scale is None else ref.d64(scale) * grads["r"], "dx")
    close(g["dw"], grads["w"], "dw")
    if gate:
        close(g["dz"], grads["z"], "dz")
    if res:
        close(g["dresidual"], grads["r"], "dresidual")
    if scaled:
        close(g["dres_scale"], (grads["r"] * ref.d64(x)).sum((0, 1, 2)), "dres_scale")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,D,N,G,state", [(257, 2048, 16, 1, True), (257, 2048, 16, 1, False), (39, 1000, 5, 2, True), (41, 600, 100, 1, True),
                                           (700, 512, 1, 1, True), (64, 2048, 16, 2, True)])
def test_scan_step_with_two_sequences_a_lane(gdn, dtype, n, D, N, G, state):
    gen = torch.Generator().manual_seed(2)
    r = lambda *s, dtype=F32, scale=1.0: (torch.randn(*s, generator=gen) * scale).to(dtype).to(DEV)  # noqa: E731
    # slices of wider projections, as in use
    x, z = r(n, 2 * D, dtype=dtype).split(D, -1)
    low = r(n, 3 + 2 * G * N, dtype=dtype)
    Bm, Cm = low[:, 3:3 + G * N].unflatten(-1, (G, N)), low[:, 3 + G * N:].unflatten(-1, (G, N))
    dt, bias, skip = r(n, D, dtype=dtype, scale=0.7), r(D, scale=0.3) - 1.5, r(D)
    A = -(0.5 + torch.rand(D, N, generator=gen) * 4).to(DEV)
    h = r(n, D, N, scale=0.5) if state else None
    v = [ref.d64(t) for t in (x, dt, A, Bm, Cm, skip, z, bias, h)]
    one = lambda t: t.unsqueeze(1)  # noqa: E731
    wy, wh = ref.scan(one(v[0]), one(v[1]), v[2], one(v[3]), one(v[4]), v[5], one(v[6]), v[7], v[8])
    y, hT = gdn.scan_step(x, dt, A, Bm, Cm, skip, z, bias, state=h)
    assert ref.err(y, wy[:, 0]) <= SCAN_TOL[dtype] and ref.err(hT, wh) <= SCAN_TOL[F32]
    last = ref.err(y[-1], wy[-1, 0])                # the sequence that has no second one beside it
    assert last <= 2 * SCAN_TOL[dtype], last
    if state:
        y2, h2 = gdn.scan_step(x, dt, A, Bm, Cm, skip, z, bias, state=h, out_state=h)
        assert h2 is h and torch.equal(y2, y) and torch.equal(h2, hT)
