"""GPU tests of what the layer calls refuse beside their tensors' types and shapes: buffers and results that the
kernels must not be given."""
import pytest
import torch

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


def calls(gdn):
    """Every call that takes a workspace, as a function of it; and the scan's backward as one of the saved buffer."""
    x, w, n = torch.ones(1, 20, 16, device=DEV), torch.ones(16, 4, device=DEV), torch.ones(16, device=DEV)
    A, B, cu = -torch.ones(16, 4, device=DEV), torch.ones(1, 20, 4, device=DEV), torch.tensor([0, 20], dtype=torch.int32, device=DEV)
    y, _, saved = gdn.scan_forward(x, x, A, B, B, save=True)
    return [lambda ws: gdn.conv_forward(x, w, cu_seqlens=cu, ws=ws), lambda ws: gdn.conv_backward(x, w, None, None, x, ws=ws),
            lambda ws: gdn.scan_forward(x, x, A, B, B, cu_seqlens=cu, ws=ws),
            lambda ws: gdn.scan_backward(x, x, A, B, B, dy=y, saved=saved, ws=ws), lambda ws: gdn.norm_backward(x, n, x, ws=ws),
            lambda ws: gdn.scan_backward(x, x, A, B, B, dy=y, saved=ws)]


@pytest.mark.parametrize("i", range(6))
def test_buffers_of_the_caller(gdn, i):
    call = calls(gdn)[i]
    room = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    call(room)
    with pytest.raises(TypeError):
        call(room.cpu())
    with pytest.raises(ValueError):
        call(room[::2])
    with pytest.raises(ValueError):
        call(room[:1].expand(1 << 20))       # one byte that claims to be many
    with pytest.raises(gdn.GdnError):
        call(room[:64])
    with pytest.raises(gdn.GdnError):
        call(room[4:])                       # not 16-byte aligned
