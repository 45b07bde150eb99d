"""GPU tests of the training operators together: a recurrent block between its residual dropout and the loss, forward and backward,
against the same chain in 64 bits (differentiated); the example's model with recurrent blocks, dropout and the loss without logits;
its single-token path; a whole training step of the operators captured into a graph.

Bounds.  float32 chain: each operator's own 1e-5 (relative Frobenius) adds up over five of them, and the norm's and the gates'
derivatives pass errors on about as they are: 1e-4.  bf16 models of different rounding places: as in the example's other test."""
import os
import sys

import pytest
import torch

import layers_ref as ref
import recur_ref

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
DEV, F32 = "cuda", torch.float32


@pytest.fixture(scope="module")
def ex():
    import __graft_entry__
    __graft_entry__.build()
    import hybrid_blocks
    return hybrid_blocks


def chain_inputs(B, T, D, V, seed=1):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k).to(DEV)  # noqa: E731
    x = dict(x=rnd(B, T, D), rg=rnd(B, T, D), ig=rnd(B, T, D), lam=rnd(D) - 3, rg_bias=rnd(D), ig_bias=rnd(D), z=rnd(B, T, D),
             residual=rnd(B, T, D), wn=rnd(D, k=0.3) + 1, w=rnd(V, D, k=D ** -0.5))
    t = torch.randint(0, V, (B, T), generator=g)
    t[0, ::7] = -100
    return x, t.to(DEV), torch.tensor([1234, 5], device=DEV)


def chain(gdn, x, t, rng, p=0.2):
    """recurrence -> dropout into the residual -> norm -> loss; losses and all gradients of their mean."""
    y, _, saved = gdn.recur_forward(x["x"], x["rg"], x["ig"], x["lam"], x["rg_bias"], x["ig_bias"], x["z"], want_state=False, save=True)
    r = gdn.dropout_forward(y, p, rng, residual=x["residual"])
    u = gdn.norm_forward(r, x["wn"])
    loss, lse = gdn.xent_forward(u, x["w"], t, check_status=False)
    g = gdn.xent_backward(u, x["w"], t, lse, torch.full((), 1.0 / t.numel(), device=DEV).expand(t.shape), check_status=False)
    n = gdn.norm_backward(r, x["wn"], g["dx"])
    dy = gdn.dropout_backward(n["dx"], p, rng)
    b = gdn.recur_backward(x["x"], x["rg"], x["ig"], x["lam"], x["rg_bias"], x["ig_bias"], x["z"], dy=dy, saved=saved)
    return loss, dict(w=g["dw"], wn=n["dw"], residual=n["dx"], x=b["dx"], rg=b["drg"], ig=b["dig"], lam=b["dlam"], rg_bias=b["drg_bias"],
                      ig_bias=b["dig_bias"], z=b["dz"])


def test_chain_against_64_bits(ex):
    gdn = ex.gdn
    x, t, rng = chain_inputs(2, 75, 48, 130)
    loss, got = chain(gdn, x, t, rng)
    v = {k: ref.d64(a).requires_grad_() for k, a in x.items()}
    y, _ = recur_ref.recur(v["x"], v["rg"], v["ig"], v["lam"], v["rg_bias"], v["ig_bias"], v["z"])
    r = recur_ref.dropout(y, 0.2, 1234, 5, v["residual"])
    u = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-6) * v["wn"]
    want = torch.nn.functional.cross_entropy((u @ v["w"].t()).flatten(0, 1), t.cpu().flatten(), ignore_index=-100, reduction="none").view(t.shape)
    (want.sum() / t.numel()).backward()
    assert ref.err(loss, want) <= 1e-5
    for k, g in got.items():
        e = ref.err(g, v[k].grad)
        assert e <= 1e-4, (k, e)


def test_chain_in_a_graph(ex):
    """The whole step captured, replayed with new inputs and a new call number: the bits of the calls."""
    gdn = ex.gdn
    a, ta, ra = chain_inputs(2, 40, 64, 90, 2)
    b, tb, rb = chain_inputs(2, 40, 64, 90, 3)
    rb[1] = 77
    want = [chain(gdn, *k) for k in ((a, ta, ra), (b, tb, rb))]
    slot, t, r = {k: v.clone() for k, v in a.items()}, ta.clone(), ra.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(gdn, slot, t, r)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, got = chain(gdn, slot, t, r)
    for (x, tt, rr), (wl, wg) in zip(((a, ta, ra), (b, tb, rb)), want):
        for k in slot:
            slot[k].copy_(x[k])
        t.copy_(tt)
        r.copy_(rr)
        graph.replay()
        assert torch.equal(loss, wl) and all(torch.equal(got[k], wg[k]) for k in wg)


def test_the_model_trains_and_every_parameter_has_a_gradient(ex):
    torch.manual_seed(0)
    model = ex.HybridModel(recurrent=1, dropout=0.1).cuda()
    losses = ex.train(model, steps=3, n=4, T=64, logits=False)
    assert all(v == v for v in losses)
    assert not [n for n, p in model.named_parameters() if p.grad is None or not bool(torch.isfinite(p.grad).all())]
    assert int(model.rng[1]) == 3 * len(model.blocks)      # a mask of its own for every call


def test_the_loss_without_logits_is_the_loss(ex):
    """Both from the same bf16 hidden states and weights: the logits of one are rounded to bf16 (half a step 2^-8 of up to some ten),
    of the other not."""
    torch.manual_seed(1)
    model = ex.HybridModel(recurrent=2).cuda()
    tokens = ex.batch(4, 50, 64, torch.Generator().manual_seed(3))
    one = model.loss(tokens)
    two = torch.nn.functional.cross_entropy(model(tokens[:, :-1]).float().flatten(0, 1), tokens[:, 1:].flatten())
    top = float(model(tokens[:, :-1]).detach().float().abs().max())
    assert abs(float(one.detach()) - float(two.detach())) <= 2 * top * 2.0 ** -8
    ga, gb = (torch.autograd.grad(v, model.blocks[-1].lam)[0] for v in (one, two))
    assert float((ga - gb).norm()) <= 0.1 * float(gb.norm())


def test_single_tokens_give_the_sequence(ex):
    torch.manual_seed(1)
    model = ex.HybridModel(pairs=1, recurrent=2).cuda().eval()
    tokens = ex.batch(3, 40, 64, torch.Generator().manual_seed(2))
    with torch.no_grad():
        whole = model(tokens).float()
    states = model.start(3)
    single = torch.stack([model.step(tokens[:, t], states).float() for t in range(tokens.shape[1])], 1)
    # bf16 between every two operators, rounded at other places in the two paths: some ten roundings of 2^-8 deep
    assert float((single - whole).norm() / whole.norm()) < 0.04
