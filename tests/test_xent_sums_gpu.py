"""GPU tests of the loss where all products of a logit have one sign: x and w around 1, so that a logit of K features is about K and what
its sum loses shows.  Forward and backward have to lose the same: a probability is exp of the difference of the backward's logit and the
forward's lse.

What a sum loses.  The tensor core cuts what it adds off: a step of 16 products loses up to 2^-23 of the sum so far (one unit u of its
last place), half of that on average, and what differs from logit to logit is a random walk of n steps of u / sqrt(12).  n = K / 16; the
sum so far is at most S = K up to 2048 features, and 1024 in segments above.  On the CUDA cores it is rounded, far less."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture()
def gdn():
    import __graft_entry__
    __graft_entry__.build()
    import chunkwise_delta_rule_02_gb300 as g
    return g


def make(M, K, V, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(M, K, generator=g) * 0.5 + 1).to(dtype).to(DEV)
    w = (torch.randn(V, K, generator=g) * 2 * K ** -0.5 + 1).to(dtype).to(DEV)
    return x, w, torch.randint(0, V, (M,), generator=g).to(DEV), torch.randn(M, generator=g).to(DEV)


#: tokens, features, entries, type, whether the call goes without the tensor cores
CASES = [(300, 9001, 200, BF, False), (40, 9001, 200, BF, False), (16, 4001, 300, BF, False), (300, 2056, 500, BF, False), (2, 9001, 200, BF, False),
         (300, 2048, 500, BF, False), (12, 1591, 500, BF, False), (7, 2047, 300, BF, False), (12, 2048, 300, BF, False), (4, 2048, 300, BF, False),
         (4, 2047, 300, BF, True), (12, 501, 300, BF, True), (300, 4001, 200, F32, False), (12, 1500, 300, F32, True)]


@pytest.mark.parametrize("M,K,V,dtype,few", CASES)
def test_gradients_of_logits_with_a_common_part(gdn, M, K, V, dtype, few):
    """By element.  D is off by the result's half step (bf16; not where the call goes without the tensor cores) and by the probability's error: 5
    times the random walk above, and 4 |lse| 2^-24 for lse, its two terms and the logit, all float32 numbers.  Then sums of at most max(M, V) terms in
    float32, cut off or rounded, 2^-23 of the terms' size a step, and the result's rounding."""
    x, w, t, dloss = make(M, K, V, dtype)
    _, lse = gdn.xent_forward(x, w, t)
    g = gdn.xent_backward(x, w, t, lse, dloss)
    logits = x.double() @ w.double().t()
    want = torch.logsumexp(logits, 1)
    d = torch.exp(logits - want[:, None])
    terms = d.clone()
    d[torch.arange(M, device=DEV), t] -= 1
    terms[torch.arange(M, device=DEV), t] += 1
    d, terms = d * dloss.double()[:, None], terms * dloss.double().abs()[:, None]
    n, S = K / 16, min(K, 1024 if K > 2048 or dtype is F32 else 2048)
    walk = 0.0 if few else 5 * n ** 0.5 * 2.0 ** -23 * 1.5 * S / 12 ** 0.5
    off = (2.0 ** -9 if dtype is BF and not few else 0.0) + walk + (4 * float(want.abs().max()) + 2 * max(M, V)) * 2.0 ** -24
    step = torch.finfo(dtype).eps / 2
    for n, ref, size in (("dx", d @ w.double(), terms @ w.double().abs()), ("dw", d.t() @ x.double(), terms.t() @ x.double().abs())):
        worst = float(((g[n].double() - ref).abs() / (off * size + step * ref.abs())).max())
        assert worst <= 1, (n, worst)


@pytest.mark.parametrize("M", [40, 300])
def test_losses_of_many_features_of_one_sign(gdn, M):
    """lse of 9001 features: nine segments of at most 64 steps.  A segment's sum grows to 1024, so that a step loses half of 2^-14 or less, over
    a segment's growth 2 / 3 of that on average: 576 steps of 2.0e-5 are 1.2e-2; 1.5 times that, and half a step 2^-10 for each of the nine
    additions and for lse, is the bound, 2.3e-2.  One sum of 563 steps up to 9001 would lose 0.11 at half a step
    each; measured with the segments switched off it loses 0.28, with them 9.2e-3."""
    x, w, t, _ = make(M, 9001, 200, BF, 2)
    _, lse = gdn.xent_forward(x, w, t)
    want = torch.logsumexp(x.double() @ w.double().t(), 1)
    assert abs(float((lse.double() - want).mean())) <= 1.5 * 1.2e-2 + 10 * 2.0 ** -11


def test_a_long_sum_over_the_vocabulary(gdn):
    """dx of 131072 entries whose weights are around 1 / 4: the positive terms, D w of all entries but the target's, grow to a sum that the tensor
    core cuts off, which the target's term then takes away.  Each of n products loses what lies 2 bits below u, 2^-27 of the sum so far on
    average, in all n 2^-28 of the terms (9001 features of one sign, one sum: 3.1e-5 against 3.4e-5): in parts of 16384 that is 6.1e-5 of the
    terms, and 1.5 times that the bound; in one of 65536 it would be 2.4e-4 (measured 2.0e-4).  D's rounding, 2^-9 each, is a random one: 1e-6."""
    M, K, V = 1024, 1024, 131072
    g = torch.Generator(device=DEV).manual_seed(3)
    x = (torch.randn(M, K, generator=g, device=DEV) * 0.3 + 1).to(BF)
    w = (torch.randn(V, K, generator=g, device=DEV) * 0.3 * K ** -0.5 + 0.25).to(BF)
    t = torch.randint(0, V, (M,), generator=g, device=DEV)
    _, lse = gdn.xent_forward(x, w, t)
    dx = gdn.xent_backward(x, w, t, lse, torch.ones((), device=DEV).expand(M))["dx"]
    d = x.double() @ w.double().t()
    d = torch.exp(d - torch.logsumexp(d, 1, keepdim=True))
    d[torch.arange(M, device=DEV), t] -= 1
    off = dx.double() - d @ w.double()
    terms = float((d.abs() @ w.double().abs()).mean())
    assert abs(float(off.mean())) <= 1.5 * 16384 * 2.0 ** -28 * terms


@pytest.mark.parametrize("M,K,V,dtype", [(4096, 24, 70001, BF), (4096, 21, 70001, BF), (2048, 520, 90000, BF), (40000, 72, 5000, BF), (700, 40, 70001, F32)])
def test_pieces_whose_products_are_cut(gdn, M, K, V, dtype):
    """Several pieces of the vocabulary (or one), each product's contraction in several parts: relative Frobenius, D and the result rounded to bf16
    once each, 2^-8 at most; float32 1e-5; and 4 max |lse| 2^-24 for the probabilities."""
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(M, K, generator=g, device=DEV).to(dtype)
    w = (torch.randn(V, K, generator=g, device=DEV) * 2 * K ** -0.5).to(dtype)
    t = torch.randint(0, V, (M,), generator=g, device=DEV)
    dloss = torch.randn(M, generator=g, device=DEV)
    _, lse = gdn.xent_forward(x, w, t)
    got = gdn.xent_backward(x, w, t, lse, dloss)
    d = x.double() @ w.double().t()
    want = torch.logsumexp(d, 1)
    d = d.sub_(want[:, None]).exp_()
    d[torch.arange(M, device=DEV), t] -= 1
    d *= dloss.double()[:, None]
    tol = (2.0 ** -8 if dtype is BF else 1e-5) + 4 * float(want.abs().max()) * 2.0 ** -24
    for n, ref in (("dx", d @ w.double()), ("dw", d.t() @ x.double())):
        assert float((got[n].double() - ref).norm() / ref.norm()) <= tol, n
    again = gdn.xent_backward(x, w, t, lse, dloss)
    assert torch.equal(got["dx"], again["dx"]) and torch.equal(got["dw"], again["dw"])
