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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_convolution_results_over_its_inputs(gdn, dtype):
    """Tokens would be read after they were written over: refused.  Another slice of the same projection is not."""
    B, H, T, d = 2, 3, 50, 16
    C = H * d
    wide = torch.randn(B, T, 3 * C, device=DEV).to(dtype)
    x, z, rest = wide.split(C, -1)
    w, state = torch.randn(C, 4, device=DEV), torch.zeros(B, 3, C, dtype=dtype, device=DEV)
    dy = torch.randn(B, T, C, device=DEV).to(dtype)
    by_head = lambda t: t.unflatten(-1, (H, d)).transpose(1, 2)  # noqa: E731
    for out in (x, wide[..., 8:8 + C], wide[:, :, C - 1:2 * C - 1]):
        with pytest.raises(ValueError):
            gdn.conv_forward(x, w, out=out)
        with pytest.raises(ValueError):
            gdn.conv_forward(by_head(x), w, out=by_head(out))
        with pytest.raises(ValueError):
            gdn.conv_backward(dy, w, None, None, x, out=out)
        with pytest.raises(ValueError):
            gdn.conv_backward(x, w, None, None, dy, out=out)
    with pytest.raises(ValueError):
        gdn.conv_forward(x[:, :3], w, state=state, out=state)
    with pytest.raises(ValueError):
        gdn.conv_backward(x[:, :3], w, None, state, dy[:, :3], state, out=state)
    with pytest.raises(ValueError):
        gdn.conv_backward(x[:, :3], w, None, None, dy[:, :3], state, out=state)
    want, _ = gdn.conv_forward(x, w)
    grad = gdn.conv_backward(x, w, None, None, dy)["dx"]
    assert torch.equal(gdn.conv_forward(x, w, out=z)[0], want) and torch.equal(z, want)
    assert torch.equal(gdn.conv_backward(x, w, None, None, dy, out=rest)["dx"], grad) and torch.equal(rest, grad)


def test_malformed_arguments_raise_the_documented_errors(gdn):
    x, w = torch.ones(1, 20, 16, device=DEV), torch.ones(16, 4, device=DEV)
    A, B = -torch.ones(16, 4, device=DEV), torch.ones(1, 20, 4, device=DEV)
    empty = torch.zeros(0, dtype=torch.int32, device=DEV)
    for f, e in ((lambda: gdn.conv_step(x[0], w[:, 0]), ValueError), (lambda: gdn.conv_step(x[0], w[:, :0]), ValueError),
                 (lambda: gdn.conv_forward(x, w[:, :0]), ValueError), (lambda: gdn.conv_forward(x, w[:, 0]), ValueError),
                 (lambda: gdn.conv_forward(x, w, cu_seqlens=empty), TypeError),
                 (lambda: gdn.conv_forward(x, w, cu_seqlens=[0, 20]), TypeError),
                 (lambda: gdn.conv_backward(x, w, None, None, x, cu_seqlens=empty), TypeError),
                 (lambda: gdn.scan_forward(x, x, A, B, B, cu_seqlens=empty), TypeError),
                 (lambda: gdn.scan_forward(x, x, A, B, B, cu_seqlens=(0, 20)), TypeError)):
        with pytest.raises(e):
            f()


def test_residual_gradients_without_a_scale_are_one_tensor(gdn):
    """As documented: equal gradients under two names; with a scale, two tensors."""
    x, w, dy = (torch.randn(3, 5, 32, device=DEV) for _ in range(3))
    g = gdn.norm_backward(x, w[0, 0], dy, sum=x)
    assert g["dx"] is g["dresidual"]
    g = gdn.norm_backward(x, w[0, 0], dy, sum=x, res_scale=torch.full((32,), 2.0, device=DEV))
    assert g["dx"].data_ptr() != g["dresidual"].data_ptr() and torch.equal(g["dx"], 2 * g["dresidual"])
