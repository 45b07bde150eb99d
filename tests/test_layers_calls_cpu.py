"""Records that the layer calls hand to the library, read by a stand-in for it (no GPU)."""
import types

import pytest
import torch


@pytest.fixture()
def lay(monkeypatch):
    from chunkwise_delta_rule_02_gb300 import layers
    calls = []

    def take(*args):
        calls.append(args)
        return 0

    monkeypatch.setattr(layers, "_lib", types.SimpleNamespace(dn_conv_step=take))
    return layers, calls


@pytest.mark.parametrize("n,C,wide", [(3, 8, 8), (2, 8, 20), (1, 5, 5)])
def test_conv_step_records_step_from_sequence_to_sequence(lay, n, C, wide):
    """One token a sequence as [n,C]: the batch stride is the row's, as for the same tokens given as [n,1,C] or [n,H,1,d]."""
    layers, calls = lay
    x, y = torch.zeros(n, wide)[:, :C], torch.zeros(n, C)
    w, bias, state = torch.zeros(C, 4), torch.zeros(C), torch.zeros(n, 3, C)
    shape = layers._CONV_SHAPE.pack(n, 1, 1, C, 4, 0, 1, 0, 0)
    for xs, ys in ((x, y), (x.unsqueeze(1), y.unsqueeze(1)), (x[:, None, None], y[:, None, None])):
        layers.dn_conv_step(shape, xs, w, bias, state, state, ys, stream=0)
        got = calls.pop()
        (px, bx, _, _), (py, by, _, _) = layers._VIEW.unpack(got[1]), layers._VIEW.unpack(got[6])
        assert (px, bx) == (x.data_ptr(), wide) and (py, by) == (y.data_ptr(), C)
        assert got[0] == shape and got[2:6] == (w.data_ptr(), bias.data_ptr(), state.data_ptr(), state.data_ptr())


def test_buffers_are_cuda_tensors():
    from chunkwise_delta_rule_02_gb300 import layers
    with pytest.raises(TypeError):
        layers._buffer(torch.zeros(256, dtype=torch.uint8), "ws", torch.zeros(1))
