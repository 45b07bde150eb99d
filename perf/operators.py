"""The layer operators around the delta rule: what is computed, on which inputs, and how much work that is.

Three operators, each with the directions that training and serving need:

* ``conv``  the short causal convolution ahead of q, k, v or of the scan's input (forward, backward, one token);
* ``scan``  the selective state space scan (forward, forward with backward, one token);
* ``norm``  the RMS norm with its output gate, or with the residual sum in front of it (forward, backward).

``run`` computes a case in plain torch operations in 32 bits, or, where ``own`` is true, through the package's calls.
Sizes come from the package's own workloads: 16 heads of 128 features, 4 x 8192 tokens for prompts, 8 x 4096 for
training, 256 sequences for single tokens, 8 packed sequences; the odd ones stand for ragged batches.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# ------------------------------------------------------------------ cases


def listed():
    return [
        # convolution of one of q, k, v for a batch of prompts: token-major projection in, head-major out
        dict(name="conv_fwd_prompt", op="conv_fwd", type="bf16", B=4, H=16, T=8192, d=128, W=4, silu=True, packed=0, state=False),
        # the same in training, forward inputs given
        dict(name="conv_bwd_train", op="conv_bwd", type="bf16", B=8, H=16, T=4096, d=128, W=4, silu=True, packed=0, state=False),
        # packed ragged sequences continuing from cached taps, float32, an odd width
        dict(name="conv_bwd_packed", op="conv_bwd", type="f32", B=1, H=5, T=9001, d=100, W=3, silu=True, packed=8, state=True),
        # one token for each of 256 sequences being served
        dict(name="conv_step", op="conv_step", type="bf16", B=256, H=16, T=1, d=128, W=4, silu=True, packed=0, state=True),
        # a batch of prompts through the scan, with its gate
        dict(name="scan_fwd_prompt", op="scan_fwd", type="bf16", B=4, T=8192, D=2048, N=16, G=1, packed=0, state=False, gate=True),
        # one long prompt in pieces: few channels, a long axis, continuing from a state
        dict(name="scan_fwd_long", op="scan_fwd", type="bf16", B=1, T=16384, D=1024, N=16, G=1, packed=0, state=True, gate=True),
        # a training step: forward and backward
        dict(name="scan_train", op="scan_train", type="bf16", B=8, T=4096, D=2048, N=16, G=1, packed=0, state=False, gate=True),
        # packed ragged sequences, float32, no gate, more states in shared groups
        dict(name="scan_train_packed", op="scan_train", type="f32", B=1, T=3001, D=640, N=32, G=2, packed=8, state=True, gate=False),
        # one token for each of 256 sequences being served
        dict(name="scan_step", op="scan_step", type="bf16", B=256, T=1, D=2048, N=16, G=1, packed=0, state=True, gate=True),
        # after a delta rule block: norm and gate per head, head-major in, token-major out
        dict(name="norm_gate_fwd", op="norm_fwd", type="bf16", B=4, H=16, T=8192, d=128, gate=True, residual=False),
        # the same in training
        dict(name="norm_gate_bwd", op="norm_bwd", type="bf16", B=8, H=16, T=4096, d=128, gate=True, residual=False),
        # before a block while serving: residual sum, scale and norm of one token for each of 256 sequences
        dict(name="norm_residual_step", op="norm_fwd", type="bf16", B=256, H=1, T=1, d=2048, gate=False, residual=True),
    ]


#: No drawn case has more (token, channel, state) elements than the largest listed one.
_MOST_SCAN = 8 * 4096 * 2048 * 16
_MOST_ROW = 4 * 8192 * 2048


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_train", "scan_step", "norm_fwd", "norm_bwd"])
    c = dict(op=op, type=rng.choice(["bf16", "bf16", "f32"]))
    if op.startswith("scan"):
        c["N"] = rng.choice([4, 8, 16, 16, 16, 32, 64])
        c["G"] = rng.choice([1, 1, 2])
        c["D"] = c["G"] * rng.choice([8, 1]) * _log(rng, 16, 128)
        if c["D"] < 96:
            c["D"] *= 8
        c["gate"] = rng.random() < 0.7
        c["state"] = rng.random() < 0.5
        if op == "scan_step":
            c.update(B=_log(rng, 1, 512), T=1, packed=0, state=True)
        else:
            most = _MOST_SCAN // (c["D"] * c["N"])
            c["packed"] = rng.choice([0, 0, 0, 3, 9])
            c["B"] = 1 if c["packed"] else _log(rng, 1, 8)
            c["T"] = _log(rng, 64, max(64, min(12000, most // (c["B"]))))
    elif op.startswith("conv"):
        c.update(H=rng.choice([1, 4, 7, 16]), d=rng.choice([64, 128, 128, 100, 129]), W=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.8)
        c["state"] = rng.random() < 0.5
        if op == "conv_step":
            c.update(B=_log(rng, 1, 512), T=1, packed=0, state=True)
        else:
            c["packed"] = rng.choice([0, 0, 0, 3, 9])
            c["B"] = 1 if c["packed"] else _log(rng, 1, 8)
            c["T"] = _log(rng, 32, min(16384, _MOST_ROW // (c["B"] * c["H"] * c["d"])))
    else:
        c["residual"] = rng.random() < 0.5
        c["gate"] = not c["residual"]
        if c["residual"]:
            c.update(H=1, d=rng.choice([1024, 2048, 2048, 4096, 1000, 2050]))
        else:
            c.update(H=rng.choice([1, 4, 7, 16]), d=rng.choice([64, 128, 128, 256, 100, 129]))
        c["B"] = _log(rng, 1, 64)
        c["T"] = _log(rng, 1, min(8192, _MOST_ROW // (c["B"] * c["H"] * c["d"])))
    return c


def _lengths(T, n, seed):
    """n ragged lengths that sum to T; the second of more than three is empty, the last one token where there is room."""
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(n, generator=g) + 0.05
    if n > 3:
        w[1] = 0.0
    lens = (w / w.sum() * T).floor().long()
    lens[0] += T - lens.sum()
    if n > 3 and lens[0] + lens[-1] > 1:
        lens[0] += lens[-1] - 1
        lens[-1] = 1
    return lens.tolist()


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = TYPES[case["type"]]

    def normal(*shape, scale=1.0, of=None):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(of or dt)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=g, device=DEV) * (hi - lo) + lo

    op = case["op"]
    s = dict(case=case, op=op)
    B, T = case["B"], case["T"]
    if case.get("packed"):
        lens = _lengths(T, case["packed"], seed)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["longest"], N = max(lens), len(lens)
    else:
        s["cu"], s["longest"], N = None, T, B
    if op.startswith("conv"):
        H, d, W = case["H"], case["d"], case["W"]
        C = H * d
        s["w"], s["bias"] = normal(C, W, scale=W ** -0.5, of=torch.float32), normal(C, scale=0.1, of=torch.float32)
        s["state"] = normal(N, W - 1, C) if case["state"] else None
        if op == "conv_step":
            s["x"] = normal(B, C)
            s["out_state"] = torch.empty_like(s["state"])
            return s
        # the projection's output is token-major, the delta rule reads head-major
        s["x"] = normal(B, T, H, d).transpose(1, 2)
        if op == "conv_bwd":
            s["dy"] = normal(B, H, T, d)
            s["dstate"] = normal(N, W - 1, C) if case["state"] else None
        return s
    if op.startswith("scan"):
        D, N_, G = case["D"], case["N"], case["G"]
        s["A"] = -(torch.arange(1, N_ + 1, device=DEV).float() * uniform(D, N_, lo=0.5, hi=1.5))
        s["D"] = normal(D, scale=1.0, of=torch.float32)
        step = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus of it is the step
        s["h0"] = normal(N, D, N_, scale=0.1, of=torch.float32) if case["state"] else None
        if op == "scan_step":
            s["x"], s["dt"] = normal(B, D), normal(B, D, scale=0.5)
            s["z"] = normal(B, D) if case["gate"] else None
            s["B"], s["C"] = normal(B, G, N_), normal(B, G, N_)
            s["out_state"] = torch.empty_like(s["h0"])
            return s
        s["x"], s["dt"] = normal(B, T, D), normal(B, T, D, scale=0.5)
        # the gate is the second half of the input projection; B and C are cut from one projection behind dt's low-rank part
        s["z"] = normal(B, T, 2 * D)[:, :, D:] if case["gate"] else None
        low = 64
        both = normal(B, T, low + 2 * G * N_)
        s["B"] = both[:, :, low:low + G * N_].unflatten(2, (G, N_))
        s["C"] = both[:, :, low + G * N_:].unflatten(2, (G, N_))
        if op == "scan_train":
            s["dy"] = normal(B, T, D)
            s["dhT"] = normal(N, D, N_, scale=0.1, of=torch.float32) if case["state"] else None
        return s
    H, d = case["H"], case["d"]
    s["w"] = uniform(d, lo=0.5, hi=1.5)
    if case["residual"]:
        s["x"], s["residual"] = normal(B, T, d), normal(B, T, d, scale=3.0)
        s["scale"] = uniform(d, lo=0.1, hi=1.0)
        s["z"] = None
        if op == "norm_bwd":
            s["sum"] = (s["residual"].float() + s["scale"] * s["x"].float()).to(dt)
            s["dy"], s["dsum"] = normal(B, T, d), normal(B, T, d)
    else:
        s["x"] = normal(B, H, T, d, scale=0.3)  # the delta rule's output
        s["z"] = normal(B, T, H, d).transpose(1, 2)  # the projection's output
        s["out"] = torch.empty(B, T, H, d, dtype=dt, device=DEV).transpose(1, 2)  # what the next projection reads
        if op == "norm_bwd":
            s["dy"] = normal(B, T, H, d).transpose(1, 2)
    return s


# ------------------------------------------------------------------ one pass


def _gdn():
    import chunkwise_delta_rule_02_gb300 as gdn
    return gdn


def _scan_args(s):
    return s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"]


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    # check_status=False, as a training or serving loop has it: reading the status word of packed input would wait for the GPU
    gdn, op, c = _gdn(), s["op"], s["case"]
    if op == "conv_fwd":
        y, state = gdn.conv_forward(s["x"], s["w"], s["bias"], s["state"], cu_seqlens=s["cu"], silu=c["silu"], check_status=False)
        return dict(y=y, state=state)
    if op == "conv_bwd":
        return gdn.conv_backward(s["x"], s["w"], s["bias"], s["state"], s["dy"], s["dstate"], cu_seqlens=s["cu"], silu=c["silu"], check_status=False)
    if op == "conv_step":
        y, state = gdn.conv_step(s["x"], s["w"], s["bias"], s["state"], out_state=s["out_state"], silu=c["silu"])
        return dict(y=y, state=state)
    if op == "scan_fwd":
        y, hT = gdn.scan_forward(*_scan_args(s), h0=s["h0"], cu_seqlens=s["cu"], check_status=False)
        return dict(y=y, state=hT)
    if op == "scan_train":
        y, hT, saved = gdn.scan_forward(*_scan_args(s), h0=s["h0"], cu_seqlens=s["cu"], save=True, check_status=False)
        grads = gdn.scan_backward(*_scan_args(s), h0=s["h0"], dy=s["dy"], dhT=s["dhT"], saved=saved, cu_seqlens=s["cu"],
                                  check_status=False)
        return dict(grads, y=y, state=hT)
    if op == "scan_step":
        y, state = gdn.scan_step(*_scan_args(s), state=s["h0"], out_state=s["out_state"])
        return dict(y=y, state=state)
    if op == "norm_fwd":
        if c["residual"]:
            y, r = gdn.norm_forward(s["x"], s["w"], residual=s["residual"], res_scale=s["scale"])
            return dict(y=y, sum=r)
        return dict(y=gdn.norm_forward(s["x"], s["w"], z=s["z"], out=s["out"]))
    if c["residual"]:
        return gdn.norm_backward(s["x"], s["w"], s["dy"], sum=s["sum"], dsum=s["dsum"], res_scale=s["scale"])
    return gdn.norm_backward(s["x"], s["w"], s["dy"], z=s["z"])


def _dsilu(u):
    p = torch.sigmoid(u)
    return p * (1 + u * (1 - p))


def _sequences(s, B, T):
    """Of each token of the flat [B*T] axis its sequence, and every sequence's first token and end."""
    if s["cu"] is None:
        ends = (torch.arange(B, device=DEV) + 1) * T
        starts = ends - T
    else:
        starts, ends = s["cu"][:-1].long(), s["cu"][1:].long()
    seq = torch.searchsorted(ends, torch.arange(B * T, device=DEV), right=True)
    return seq, starts, ends


def _run_plain(s):
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[s["op"][:4]](s)


def _plain_conv(s):
    op, c, dt = s["op"], s["case"], s["x"].dtype
    w, bias = s["w"], s["bias"]
    C, W = w.shape
    act = torch.nn.functional.silu if c["silu"] else (lambda u: u)
    if op == "conv_step":
        taps = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
        y = act((taps * w.t()).sum(1) + bias).to(dt)
        s["out_state"].copy_(taps[:, 1:])
        return dict(y=y, state=s["out_state"])
    B, H, T, d = s["x"].shape
    seq, starts, ends = _sequences(s, B, T)
    # every sequence with its W-1 earlier taps in front, one after another
    N = starts.numel()
    at = torch.arange(B * T, device=DEV) + (seq + 1) * (W - 1)
    first = starts + torch.arange(N, device=DEV) * (W - 1)
    last = ends + torch.arange(1, N + 1, device=DEV) * (W - 1)
    taps = torch.arange(W - 1, device=DEV)
    rows = torch.zeros(B * T + N * (W - 1), C, device=DEV)
    rows[at] = s["x"].transpose(1, 2).reshape(B * T, C).float()
    if s["state"] is not None:
        rows[first[:, None] + taps] = s["state"].float()
    pre = bias + sum(rows[at - (W - 1) + k] * w[:, k] for k in range(W))
    heads = lambda v: v.view(B, T, H, d).transpose(1, 2).to(dt).contiguous()  # noqa: E731
    end = last[:, None] - (W - 1) + taps
    if op == "conv_fwd":
        return dict(y=heads(act(pre)), state=rows[end].to(dt))
    dpre = s["dy"].transpose(1, 2).reshape(B * T, C).float()
    if c["silu"]:
        dpre = dpre * _dsilu(pre)
    wide = torch.zeros(rows.shape[0] + W - 1, C, device=DEV)
    wide[at] = dpre
    drows = sum(wide[W - 1 - k:W - 1 - k + rows.shape[0]] * w[:, k] for k in range(W))
    if s["dstate"] is not None:
        drows.index_put_((end,), s["dstate"].float(), accumulate=True)
    dw = torch.stack([(dpre * rows[at - (W - 1) + k]).sum(0) for k in range(W)], 1)
    ds = drows[first[:, None] + taps].to(dt) if s["state"] is not None else None
    return dict(dx=drows[at].view(B, T, H, d).transpose(1, 2).to(dt), dw=dw, dbias=dpre.sum(0), dstate=ds)


def _doubling(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, in place, for sequences of at most `longest` tokens (a_t = 0 at their starts)."""
    k = 1
    while k < longest:
        b[k:] += a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _plain_scan(s):
    op, dt = s["op"], s["x"].dtype
    A, Dskip, bias = s["A"], s["D"], s["dt_bias"]
    D, N = A.shape
    G = s["B"].shape[-2]
    step = op == "scan_step"
    flat = lambda v: v.reshape(-1, D).float()  # noqa: E731
    x, raw = flat(s["x"]), flat(s["dt"]) + bias
    z = None if s["z"] is None else flat(s["z"])
    Bm, Cm = (s[k].reshape(-1, G, 1, N).float() for k in ("B", "C"))
    M = x.shape[0]
    delta = torch.nn.functional.softplus(raw)
    per = lambda v: v.view(M, G, D // G, 1)  # noqa: E731
    Ag = A.view(G, D // G, N)
    decay = torch.exp(per(delta) * Ag)
    b = per(delta * x) * Bm
    if step:
        h = decay * s["h0"].view(M, G, D // G, N) + b
        s["out_state"].copy_(h.view(M, D, N))
        y = (h * Cm).sum(-1).view(M, D) + Dskip * x
        return dict(y=(y if z is None else y * torch.nn.functional.silu(z)).to(dt), state=s["out_state"])
    shape = s["x"].shape
    seq, starts, ends = _sequences(s, shape[0], shape[1])
    full = (ends > starts).nonzero()[:, 0]
    begin, end = starts[full], ends[full] - 1
    a = decay.clone()
    a[begin] = 0
    if s["h0"] is not None:
        b[begin] += decay[begin] * s["h0"][full].view(-1, G, D // G, N)
    h = _doubling(a, b, s["longest"])
    out = (h * Cm).sum(-1).view(M, D) + Dskip * x
    hT = torch.zeros(starts.numel(), D, N, device=DEV) if s["h0"] is None else s["h0"].clone()
    hT[full] = h[end].view(-1, D, N)
    y = (out if z is None else out * torch.nn.functional.silu(z)).to(dt).view(shape)
    if op == "scan_fwd":
        return dict(y=y, state=hT)
    dy = flat(s["dy"])
    g = dy if z is None else dy * torch.nn.functional.silu(z)
    dz = None if z is None else (dy * out * _dsilu(z)).to(dt).view(shape)
    # dh_t = C_t g_t + decay_{t+1} dh_{t+1}: the same scan over the reversed axis
    dh = per(g) * Cm
    a = torch.zeros_like(decay)
    a[:-1] = decay[1:]
    a[end] = 0
    if s["dhT"] is not None:
        dh[end] += s["dhT"][full].view(-1, G, D // G, N)
    dh = _doubling(a.flip(0), dh.flip(0), s["longest"]).flip(0)
    del a
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[begin] = 0 if s["h0"] is None else s["h0"][full].view(-1, G, D // G, N)
    e = decay * before * dh
    dhB = (dh * Bm).sum(-1).view(M, D)
    ddt = ((e * Ag).sum(-1).view(M, D) + dhB * x) * torch.sigmoid(raw)
    like = s["B"].shape
    dh0 = None
    if s["h0"] is not None:
        dh0 = torch.zeros_like(s["h0"]) if s["dhT"] is None else s["dhT"].clone()
        dh0[full] = (decay[begin] * dh[begin]).view(-1, D, N)
    return dict(
        y=y, state=hT, dx=(delta * dhB + Dskip * g).to(dt).view(shape), ddt=ddt.to(dt).view(shape), dz=dz,
        dA=(per(delta) * e).sum(0).view(D, N), dD=(g * x).sum(0), ddt_bias=ddt.sum(0),
        dB=(per(delta * x) * dh).sum(2).to(dt).view(like), dC=(per(g) * h).sum(2).to(dt).view(like), dh0=dh0)


def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    x, w, eps = s["x"].float(), s["w"], 1e-6
    silu = torch.nn.functional.silu
    if s["op"] == "norm_fwd":
        r = s["residual"].float() + s["scale"] * x if c["residual"] else x
        y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + eps) * w
        if c["residual"]:
            return dict(y=y.to(dt), sum=r.to(dt))
        s["out"].copy_(y * silu(s["z"].float()))
        return dict(y=s["out"])
    r = s["sum"].float() if c["residual"] else x
    dy = s["dy"].float()
    q = torch.rsqrt(r.square().mean(-1, keepdim=True) + eps)
    gate = 1.0 if s["z"] is None else silu(s["z"].float())
    g = dy * w * gate
    dr = q * (g - r * q.square() * (g * r).mean(-1, keepdim=True))
    rest = tuple(range(r.dim() - 1))
    dw = (dy * r * q * gate).sum(rest)
    if c["residual"]:
        dr = dr + s["dsum"].float()
        return dict(dx=(s["scale"] * dr).to(dt), dw=dw, dz=None, dresidual=dr.to(dt), dres_scale=(dr * x).sum(rest))
    return dict(dx=dr.to(dt), dw=dw, dz=(dy * r * q * w * _dsilu(s["z"].float())).to(dt), dresidual=None, dres_scale=None)


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    """What ``run`` returns, in float64, token by token (scan), sequence by sequence (convolution), by differentiation (gradients of
    the convolution and the norm)."""
    s = prepare(dict(case), seed)
    for k, v in s.items():
        if isinstance(v, torch.Tensor) and v.is_floating_point():
            s[k] = v.double()
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[s["op"][:4]](s)


def _spans(s, T):
    """(batch row, first token, end, sequence) of every sequence."""
    if s["cu"] is None:
        return [(b, 0, T, b) for b in range(s["case"]["B"])]
    cu = s["cu"].tolist()
    return [(0, cu[i], cu[i + 1], i) for i in range(len(cu) - 1)]


def _exact_conv(s):
    c, w, W = s["case"], s["w"], s["case"]["W"]
    act = (lambda u: u / (1 + torch.exp(-u))) if c["silu"] else (lambda u: u)
    if s["op"] == "conv_step":
        rows = torch.cat([s["state"], s["x"][:, None]], 1)
        return dict(y=act(torch.einsum("nkc,ck->nc", rows, w) + s["bias"]), state=rows[:, 1:])
    grad = s["op"] == "conv_bwd"
    C = c["H"] * c["d"]
    leaves = {k: s[k].clone().requires_grad_(grad) for k in ("x", "w", "bias")}
    spans = _spans(s, c["T"])
    first = s["state"] if s["state"] is not None else torch.zeros(len(spans), W - 1, C, dtype=torch.float64, device=DEV)
    first = first.clone().requires_grad_(grad)
    ys, ends = [], []
    for b, lo, hi, n in spans:
        rows = torch.cat([first[n], leaves["x"][b, :, lo:hi].transpose(0, 1).reshape(hi - lo, C)])
        pre = leaves["bias"] + (rows.unfold(0, W, 1) * leaves["w"]).sum(-1) if hi > lo else rows[:0]
        ys.append(act(pre))
        ends.append(rows[rows.shape[0] - (W - 1):])
    y = torch.cat(ys).view(c["B"], c["T"], c["H"], c["d"]).transpose(1, 2)
    state = torch.stack(ends)
    if not grad:
        return dict(y=y, state=state)
    loss = (y * s["dy"]).sum()
    if s["dstate"] is not None:
        loss = loss + (state * s["dstate"]).sum()
    loss.backward()
    return dict(dx=leaves["x"].grad, dw=leaves["w"].grad, dbias=leaves["bias"].grad, dstate=first.grad if s["state"] is not None else None)


def _exact_scan(s):
    c, A = s["case"], s["A"]
    D, N = A.shape
    B, T, G = c["B"], c["T"], c["G"]
    if s["op"] == "scan_step":
        for k in ("x", "dt", "z", "B", "C"):
            s[k] = s[k].unsqueeze(1) if s[k] is not None else None
    raw = s["dt"] + s["dt_bias"]
    delta = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw)))
    wide = lambda v: v.repeat_interleave(D // G, dim=-2)  # noqa: E731
    spans = _spans(s, T)
    batched = s["cu"] is None
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(len(spans), D, N, dtype=torch.float64, device=DEV)
    starts = {lo: n for _, lo, hi, n in spans if hi > lo}
    ends = {hi - 1: n for _, lo, hi, n in spans if hi > lo}
    hT = h0.clone()
    bwd = s["op"] == "scan_train"
    kept = torch.empty(T, B, D, N, dtype=torch.float64, device=DEV) if bwd else None
    out = torch.empty(B, T, D, dtype=torch.float64, device=DEV)
    h = h0.clone() if batched else None
    for t in range(T):
        if not batched and t in starts:
            h = h0[starts[t]][None].clone()
        if bwd:
            kept[t] = h
        u = delta[:, t]
        h = torch.exp(u[..., None] * A) * h + (u * s["x"][:, t])[..., None] * wide(s["B"][:, t])
        out[:, t] = (h * wide(s["C"][:, t])).sum(-1)
        if not batched and t in ends:
            hT[ends[t]] = h[0]
    if batched:
        hT = h
    out += s["D"] * s["x"]
    gate = 1.0 if s["z"] is None else s["z"] / (1 + torch.exp(-s["z"]))
    y = out * gate
    if not bwd:
        return dict(y=y[:, 0] if s["op"] == "scan_step" else y, state=hT)
    g = s["dy"] * gate
    dz = None
    if s["z"] is not None:
        p = 1 / (1 + torch.exp(-s["z"]))
        dz = s["dy"] * out * (p + s["z"] * p * (1 - p))
    dx, ddelta = s["D"] * g, torch.empty_like(delta)
    dB, dC = torch.empty_like(s["B"]), torch.empty_like(s["C"])
    dA = torch.zeros_like(A)
    zero = torch.zeros_like(h0) if s["dhT"] is None else s["dhT"]
    dh0 = zero.clone()
    back = zero.clone() if batched else None  # what arrives at h_t from later tokens
    for t in reversed(range(T)):
        if not batched and t in ends:
            back = zero[ends[t]][None].clone()
        u, xt, Bt, Ct = delta[:, t], s["x"][:, t], wide(s["B"][:, t]), wide(s["C"][:, t])
        a = torch.exp(u[..., None] * A)
        dh = back + g[:, t][..., None] * Ct
        h = a * kept[t] + (u * xt)[..., None] * Bt
        e = dh * a * kept[t]
        dot = (dh * Bt).sum(-1)
        ddelta[:, t] = (e * A).sum(-1) + dot * xt
        dx[:, t] += u * dot
        dA += (e * u[..., None]).sum(0)
        dB[:, t] = ((u * xt)[..., None] * dh).view(B, G, D // G, N).sum(2)
        dC[:, t] = (g[:, t][..., None] * h).view(B, G, D // G, N).sum(2)
        back = a * dh
        if not batched and t in starts:
            dh0[starts[t]] = back[0]
    if batched:
        dh0 = back
    ddt = ddelta / (1 + torch.exp(-raw))
    return dict(y=y, state=hT, dx=dx, ddt=ddt, dz=dz, dA=dA, dD=(g * s["x"]).sum((0, 1)), ddt_bias=ddt.sum((0, 1)), dB=dB, dC=dC,
                dh0=dh0 if s["h0"] is not None else None)


def _exact_norm(s):
    c, grad = s["case"], s["op"] == "norm_bwd"
    names = [k for k in ("x", "w", "z", "residual", "scale", "sum") if s.get(k) is not None]
    v = {k: s[k].clone().requires_grad_(grad) for k in names}

    def normed(r):
        y = r / torch.sqrt((r * r).sum(-1, keepdim=True) / c["d"] + 1e-6) * v["w"]
        return y if s["z"] is None else y * v["z"] / (1 + torch.exp(-v["z"]))

    if not grad:
        if not c["residual"]:
            return dict(y=normed(v["x"]))
        r = v["residual"] + v["scale"] * v["x"]
        return dict(y=normed(r), sum=r)
    if not c["residual"]:
        (normed(v["x"]) * s["dy"]).sum().backward()
        return dict(dx=v["x"].grad, dw=v["w"].grad, dz=v["z"].grad, dresidual=None, dres_scale=None)
    ((normed(v["sum"]) * s["dy"]).sum() + (v["sum"] * s["dsum"]).sum()).backward()
    dr = v["sum"].grad
    ((v["scale"] * v["x"]) * dr).sum().backward()  # sum = residual + scale x
    return dict(dx=v["x"].grad, dw=v["w"].grad, dz=None, dresidual=dr, dres_scale=v["scale"].grad)


# ------------------------------------------------------------------ work


def work(case):
    op, e = case["op"], 2 if case["type"] == "bf16" else 4
    B, T = case["B"], case["T"]
    seqs = case.get("packed") or B
    if op.startswith("conv"):
        C, W = case["H"] * case["d"], case["W"]
        n, st = B * T * C, seqs * (W - 1) * C * e
        par = C * (W + 1) * 4
        if op == "conv_step":
            return dict(bytes=2 * n * e + 2 * st + par, flops=n * (2 * W + 4))
        if op == "conv_fwd":
            return dict(bytes=2 * n * e + st * (2 if case["state"] else 1) + par, flops=n * (2 * W + 4))
        return dict(bytes=3 * n * e + st * (3 if case["state"] else 0) + 2 * par, flops=n * (6 * W + 10))
    if op.startswith("scan"):
        D, N, G = case["D"], case["N"], case["G"]
        n, bc, st, par = B * T * D, B * T * G * N * e, seqs * D * N * 4, D * (N + 2) * 4
        z = 1 if case["gate"] else 0
        if op == "scan_step":
            return dict(bytes=n * e * (3 + z) + 2 * bc + 2 * st + par, flops=n * (7 * N + 10))
        if op == "scan_fwd":
            return dict(bytes=n * e * (3 + z) + 2 * bc + st * (2 if case["state"] else 1) + par, flops=n * (7 * N + 10))
        return dict(bytes=n * e * (6 + 2 * z) + 4 * bc + st * (4 if case["state"] else 1) + 2 * par, flops=n * (22 * N + 24))
    n, d = B * T * case["H"] * case["d"], case["d"]
    if op == "norm_fwd":
        return dict(bytes=n * e * (4 if case["residual"] else 3) + d * 4 * (2 if case["residual"] else 1), flops=n * 8)
    # the gate: x, z, dy in, dx, dz out; the residual: x, sum, dy, dsum in, dx, dresidual out
    return dict(bytes=n * e * (6 if case["residual"] else 5) + d * 4 * (4 if case["residual"] else 2), flops=n * 16)
