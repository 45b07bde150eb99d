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


def test_overlap_of_strided_tensors_against_their_offsets():
    """_meet says what comparing all elements' places says, for views of one buffer: slices, transposed and broadcast ones."""
    import random
    from chunkwise_delta_rule_02_gb300 import layers
    rng, room, places = random.Random(1), torch.zeros(4000), torch.arange(4000)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        views = []
        for _ in range(2):
            dims = rng.choice([1, 2, 3, 4])
            shape = [rng.randint(1, 5) for _ in range(dims)]
            if rng.random() < 0.5:      # as a slice of a dense array with its axes in some order
                order, stride, step = rng.sample(range(dims), dims), [0] * dims, 1
                for a in order:
                    stride[a] = step
                    step *= shape[a] + rng.choice([0, 0, 1, 4])
            else:
                stride = [rng.choice([0, 1, 2, 3, 7, 20, 60]) for _ in range(dims)]
            last = sum((n - 1) * st for n, st in zip(shape, stride))
            if last >= 4000:
                shape, stride, last = [3], [2], 4
            views.append((shape, stride, rng.randint(0, min(3999 - last, 300))))
        a, b = (room.as_strided(*v) for v in views)
        want = not set(places.as_strided(*views[0]).flatten().tolist()).isdisjoint(places.as_strided(*views[1]).flatten().tolist())
        assert layers._meet(a, b) == want, views
        seen[want] += 1
    assert min(seen.values()) > 300
    assert not layers._meet(room[:0], room)


def test_overlap_of_the_layouts_in_use():
    from chunkwise_delta_rule_02_gb300 import layers
    B, T, H, d = 4, 8192, 16, 128
    C = H * d
    row = 3 * C              # one projection holds x, z and something else

    def view(shape, stride, at):      # bf16 tensors too large to make here, by their places alone
        return types.SimpleNamespace(shape=shape, stride=lambda: stride, numel=lambda: 1, element_size=lambda: 2,
                                     data_ptr=lambda: (1 << 40) + at * 2)

    by_token = lambda at: view((B, T, C), (T * row, row, 1), at)                          # noqa: E731
    by_head = lambda at: view((B, H, T, d), (T * row, d, row, 1), at)                     # noqa: E731
    head_major = lambda at: view((B, H, T, d), (H * T * d, T * d, d, 1), at)              # noqa: E731
    assert not layers._meet(by_token(0), by_token(C)) and not layers._meet(by_head(C), by_token(2 * C))
    assert layers._meet(by_head(C), by_token(C)) and layers._meet(by_token(C), by_token(C + 64))
    assert layers._meet(head_major(0), by_head(0)) and layers._meet(head_major(5), by_token(C))
    assert not layers._meet(head_major(B * T * row), by_head(0)) and not layers._meet(by_head(0), head_major(B * T * row))
    assert layers._meet(view((B, T, C), (0, C, 1), 0), view((B, T, C), (T * C, C, 1), 0))
