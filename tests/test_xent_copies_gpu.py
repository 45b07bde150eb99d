"""GPU tests of the loss' copies of x and w: they hold what lies in a row and zeros, nothing of what lies behind it.  A row of 8, 24,
136 or 1592 bf16 features is 8 short of the copy's, whose rows have a multiple of 16; the inputs are views into larger arrays, so that
a read behind a row stays within one, and is found in the caller's workspace by a pattern that no logit, gradient or sum has."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
MARK = 0x7E5A            # 7.2e37 in bf16


@pytest.fixture()
def lay():
    import __graft_entry__
    __graft_entry__.build()
    from chunkwise_delta_rule_02_gb300 import layers
    return layers


def within(t, pitch):
    """t as the first columns of wider rows that hold the mark."""
    rows = t.reshape(-1, t.shape[-1])
    big = torch.full((rows.shape[0] + 1, pitch), MARK, dtype=torch.int16, device=DEV).view(BF)
    big[:-1, :t.shape[-1]] = rows
    return big


def marks(ws):
    return int((ws.view(torch.int64) == MARK * 0x0001000100010001).sum())


@pytest.mark.parametrize("K", [8, 24, 136, 1592, 16, 64])
@pytest.mark.parametrize("M,V", [(40, 300), (300, 200)])
def test_a_copy_ends_with_its_row(lay, M, V, K):
    g = torch.Generator().manual_seed(K)
    x = torch.randn(M, K, generator=g).to(BF).to(DEV)
    w = (torch.randn(1, K, generator=g) * K ** -0.5).to(BF).to(DEV)
    t, dloss = torch.randint(0, V, (M,), generator=g).to(DEV), torch.randn(M, generator=g).to(DEV)
    bx, bw = within(x, K + 8), within(w, K + 8)
    one = bw[:1, :K].expand(V, K)                                     # rows at no distance: copied
    views = [(bx[:-1, :K], one, t, dloss)]
    b3 = within(x, K + 8)[:-1].view(2, M // 2, K + 8)                 # rows at two distances: copied by the forward too
    gap = torch.full((2, M // 2 + 1, K + 8), MARK, dtype=torch.int16, device=DEV).view(BF)
    gap[:, :-1] = b3
    views.append((gap[:, :-1, :K], one, t.view(2, -1), dloss.view(2, -1)))
    for xv, wv, tv, dv in views:
        shape = lay.xent_shape(xv, wv)
        loss, lse = (torch.empty(tv.shape, device=DEV) for _ in range(2))
        ws = torch.zeros(lay.dn_xent_workspace_size(shape, xv, wv), dtype=torch.uint8, device=DEV)
        lay.dn_xent_fwd(shape, xv, wv, tv, loss, lse, ws)
        assert marks(ws) == 0
        ws = torch.zeros(lay.dn_xent_workspace_size(shape, xv, wv, True), dtype=torch.uint8, device=DEV)
        dx, dw = torch.empty(xv.shape, dtype=BF, device=DEV), torch.empty(V, K, dtype=BF, device=DEV)
        lay.dn_xent_bwd(shape, xv, wv, tv, lse, dv, dx, dw, ws)
        assert marks(ws) == 0 and lay.dn_device_status(ws) == 0
        # and the values are those of dense rows
        w2 = one.contiguous()
        loss2, lse2 = lay.xent_forward(x, w2, t)
        g2 = lay.xent_backward(x, w2, t, lse2, dloss)
        assert torch.equal(loss.flatten(), loss2) and torch.equal(dx.view(M, K), g2["dx"]) and torch.equal(dw, g2["dw"])
