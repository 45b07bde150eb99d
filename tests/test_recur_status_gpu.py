"""GPU tests of the status word of the gated linear recurrence: every call, packed or not, clears it when it starts, says in it when a
wait ran out (see test_recur_waits_gpu.py for the hooks), and writes to no other call's."""
import pytest
import torch

from test_recur_waits_gpu import CASES, INPUTS, backward, forward, make, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture()
def gdn():
    import __graft_entry__
    __graft_entry__.build()
    import chunkwise_delta_rule_02_gb300 as g
    return g


@pytest.mark.parametrize("c", [(2, 70, 64, torch.bfloat16, None), (1, 2000, 30, torch.float32, None), (1, 90, 64, torch.bfloat16, [40, 50]),
                               (2, 0, 16, torch.float32, None), (1, 33, 7, torch.float32, None)])
def test_a_call_clears_the_word(gdn, c):
    from chunkwise_delta_rule_02_gb300 import binding
    k = make(*c)
    wf, wb = workspace(k, False).fill_(255), workspace(k, True).fill_(255)
    _, saved = forward(gdn, k, wf)
    assert binding.dn_device_status(wf) == binding.DN_OK
    backward(gdn, k, saved, wb)
    assert binding.dn_device_status(wb) == binding.DN_OK


def test_a_time_out_is_forgotten_by_the_next_call(gdn, monkeypatch):
    from chunkwise_delta_rule_02_gb300 import binding
    k = make(*CASES[0])
    ws = workspace(k, False)
    monkeypatch.setenv(INPUTS, "1")
    forward(gdn, k, ws)
    monkeypatch.delenv(INPUTS)
    forward(gdn, k, ws)
    assert binding.dn_device_status(ws) == binding.DN_OK
    monkeypatch.setenv(INPUTS, "1")
    forward(gdn, k, ws)
    assert binding.dn_device_status(ws) == binding.DN_ERR_TIMEOUT


def test_no_call_writes_to_the_buffer_that_others_share(gdn, monkeypatch):
    """A convolution without packing takes the buffer; a recurrence that runs out does not touch it."""
    from chunkwise_delta_rule_02_gb300 import layers
    x = torch.randn(1, 20, 8, device="cuda")
    gdn.conv_forward(x, torch.randn(8, 4, device="cuda"))
    shared = layers._status_only[x.get_device()]
    k = make(*CASES[0])
    monkeypatch.setenv(INPUTS, "0")
    y, _ = gdn.recur_forward(*k["args"], **k["more"])
    monkeypatch.delenv(INPUTS)
    assert bool(y.isnan().any()) and not bool(shared.any())
