"""Failure detection in the gated linear recurrence, exercised without any GPU fault.

Its waits, for the inputs of a step and for the maps of a cluster's blocks, are bounded.  The test hooks GDN_DEBUG_WITHHOLD_INPUTS=n and
GDN_DEBUG_WITHHOLD_MAP=n have step n wait for 16 bytes that nobody sends, and with either set a wait gives up after about a millisecond.  The call
then ends, the workspace's status word says DN_ERR_TIMEOUT, and every result is either what it is without the hook, to the bit, or
NaN: nothing that looks like a value is made of what was not there.  The next call is right."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
INPUTS, MAP = "GDN_DEBUG_WITHHOLD_INPUTS", "GDN_DEBUG_WITHHOLD_MAP"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture()
def gdn():
    import chunkwise_delta_rule_02_gb300 as g
    return g


def make(B, T, D, dtype, lens, seed=1):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, dt=F32: torch.randn(*s, generator=g).to(dt).to(DEV)  # noqa: E731
    n = B if lens is None else len(lens)
    cu = None if lens is None else torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)
    return dict(args=(*(rnd(B, T, D, dt=dtype) for _ in range(3)), rnd(D) - 4), more=dict(z=rnd(B, T, D, dt=dtype), h0=rnd(n, D), cu_seqlens=cu),
                dy=rnd(B, T, D, dt=dtype), dhT=rnd(n, D))


def forward(gdn, k, ws):
    y, hT, saved = gdn.recur_forward(*k["args"], **k["more"], save=True, ws=ws, check_status=False)
    return dict(y=y, hT=hT), saved


def backward(gdn, k, saved, ws):
    g = gdn.recur_backward(*k["args"], **k["more"], dy=k["dy"], dhT=k["dhT"], saved=saved, ws=ws, check_status=False)
    return {n: t for n, t in g.items() if t is not None}


def workspace(k, bwd):
    from chunkwise_delta_rule_02_gb300 import layers
    n = layers.dn_recur_workspace_size(layers.recur_shape(k["args"][0], 8.0, k["more"]["cu_seqlens"]), bwd)
    return torch.zeros(n, dtype=torch.uint8, device=DEV)


#: rows enough that blocks are alone (6 steps and more), clusters of several blocks (3 steps and more), packed ones; widths that come by TMA
CASES = [(40, 700, 256, BF, None), (160, 800, 40, F32, None), (1, 9300, 64, BF, None), (1, 5000, 40, F32, None),
         (1, 9300, 64, BF, [4000, 0, 1, 5299]), (1, 2000, 10000, F32, [5, 1200, 795])]


def run_out(gdn, k, name, step, monkeypatch):
    from chunkwise_delta_rule_02_gb300 import binding
    wf, wb = workspace(k, False), workspace(k, True)
    want, saved = forward(gdn, k, wf)
    grads = backward(gdn, k, saved, wb)
    assert binding.dn_device_status(wf) == binding.dn_device_status(wb) == binding.DN_OK
    seen = []
    for call, ref, ws in ((lambda: forward(gdn, k, wf)[0], want, wf), (lambda: backward(gdn, k, saved, wb), grads, wb)):
        monkeypatch.setenv(name, str(step))
        t0 = time.perf_counter()
        got = call()
        status = binding.dn_device_status(ws)
        assert time.perf_counter() - t0 < 5.0
        monkeypatch.delenv(name)
        wrong = [n for n in ref if not bool(((got[n] == ref[n]) | got[n].isnan()).all())]
        assert not wrong, wrong
        lost = any(bool(t.isnan().any()) for t in got.values())
        assert lost == (status == binding.DN_ERR_TIMEOUT) and status in (binding.DN_OK, binding.DN_ERR_TIMEOUT)
        assert binding.dn_device_status(ws) == binding.DN_OK                # reading clears it
        again = call()
        assert all(torch.equal(again[n], ref[n]) for n in ref) and binding.dn_device_status(ws) == binding.DN_OK
        seen.append(lost)
    return seen


@pytest.mark.parametrize("step", [0, 1, 2])
@pytest.mark.parametrize("c", CASES)
def test_inputs_that_do_not_come(gdn, c, step, monkeypatch):
    assert run_out(gdn, make(*c), INPUTS, step, monkeypatch) == [True, True]


@pytest.mark.parametrize("step", [0, 1, 2])
@pytest.mark.parametrize("c", CASES[2:5] + [(1, 9300, 63, BF, None)])
def test_maps_that_do_not_come(gdn, c, step, monkeypatch):
    assert run_out(gdn, make(*c), MAP, step, monkeypatch) == [True, True]


def test_a_step_that_a_call_does_not_have_changes_nothing(gdn, monkeypatch):
    assert run_out(gdn, make(*CASES[0]), INPUTS, 1000, monkeypatch) == [False, False]
    assert run_out(gdn, make(*CASES[0]), MAP, 0, monkeypatch) == [False, False]
