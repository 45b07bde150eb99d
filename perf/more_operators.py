"""What training and serving a hybrid stack needs around its blocks: what is computed, on which inputs, and how much work that is.

Three operators, each with the directions that training and serving need:

* ``recur``  the gated linear recurrence, one state a channel, its decay and input gates in the pass (forward, forward with backward, one token);
* ``xent``   the softmax cross entropy of the last hidden states against an output weight, without keeping the logits (forward, forward with backward);
* ``drop``   dropout by a counter-based generator, with the residual's addition (forward, backward).

``run`` computes a case in plain torch operations in 32 bits, or, where ``own`` is true, through the package's calls.
Sizes come from the package's own workloads (4 x 8192 tokens for prompts, 8 x 4096 for training, 256 sequences for single
tokens, 16 heads of 128 features, 8 packed sequences) and a generic vocabulary of 2^15; the odd ones stand for ragged batches.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
IGNORE = -100      # a target without a loss
DECAY = 8.0        # the recurrence's c: log a = -c softplus(lam) sigmoid(gate)

# ------------------------------------------------------------------ cases


def listed():
    return [
        # a batch of prompts through a recurrent block, with its output gate
        dict(name="recur_fwd_prompt", op="recur_fwd", type="bf16", B=4, T=8192, D=2048, packed=0, state=False, gate=True),
        # one long prompt in pieces: few channels, a long axis, continuing from a state
        dict(name="recur_fwd_long", op="recur_fwd", type="bf16", B=1, T=16384, D=1024, packed=0, state=True, gate=False),
        # a training step: forward and backward
        dict(name="recur_train", op="recur_train", type="bf16", B=8, T=4096, D=2048, packed=0, state=False, gate=True),
        # packed ragged sequences, float32, an odd width, continuing from states
        dict(name="recur_train_packed", op="recur_train", type="f32", B=1, T=9001, D=501, packed=8, state=True, gate=False),
        # one token for each of 256 sequences being served
        dict(name="recur_step", op="recur_step", type="bf16", B=256, T=1, D=2048, packed=0, state=True, gate=True),
        # scoring a handful of tokens: the weight is read once
        dict(name="xent_score", op="xent_fwd", type="bf16", M=7, K=2048, V=32768),
        # scoring one prompt: its log likelihood
        dict(name="xent_fwd_prompt", op="xent_fwd", type="bf16", M=8192, K=2048, V=32768),
        # a training step over one sequence batch: loss, gradients of the hidden states and of the weight
        dict(name="xent_train", op="xent_train", type="bf16", M=8192, K=2048, V=32768),
        # a small model in float32, all sizes odd
        dict(name="xent_train_odd", op="xent_train", type="f32", M=1001, K=203, V=5003),
        # a block's output dropped into the residual stream, prompt-sized batch
        dict(name="drop_residual", op="drop_fwd", type="bf16", B=4, T=8192, d=2048, residual=True),
        # the same in training, gradient
        dict(name="drop_bwd", op="drop_bwd", type="bf16", B=8, T=4096, d=2048, residual=False),
        # a ragged float32 batch without a residual
        dict(name="drop_odd", op="drop_fwd", type="f32", B=3, T=1001, d=1001, residual=False),
    ]


#: No drawn case has more elements (recur, drop), or more multiply-adds (xent), than the largest listed one.
_MOST = 4 * 8192 * 2048
_MOST_MADS = 8192 * 2048 * 32768


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["recur_fwd", "recur_train", "recur_train", "recur_step", "xent_fwd", "xent_train", "xent_train", "drop_fwd", "drop_bwd"])
    c = dict(op=op, type=rng.choice(["bf16", "bf16", "f32"]))
    if op.startswith("recur"):
        c.update(D=rng.choice([1, 1, 8, 8]) * _log(rng, 16, 512), gate=rng.random() < 0.6, state=rng.random() < 0.5)
        if op == "recur_step":
            c.update(B=_log(rng, 1, 512), T=1, packed=0, state=True)
        else:
            c["packed"] = rng.choice([0, 0, 0, 3, 9])
            c["B"] = 1 if c["packed"] else _log(rng, 1, 8)
            c["T"] = _log(rng, 32, min(16384, _MOST // (c["B"] * c["D"])))
    elif op.startswith("xent"):
        most = _MOST_MADS // (8 if c["type"] == "f32" else 1)
        c["K"] = _log(rng, 64, 4096)
        c["V"] = _log(rng, 100, 131072)
        c["M"] = _log(rng, 1, min(16384, max(1, most // (c["K"] * c["V"]))))
        while c["M"] * c["K"] * c["V"] > most:
            c["V"] //= 2
    else:
        c.update(d=rng.choice([1, 1, 8]) * _log(rng, 16, 512), residual=op == "drop_fwd" and rng.random() < 0.6)
        c["B"] = _log(rng, 1, 16)
        c["T"] = _log(rng, 8, min(8192, _MOST // (c["B"] * c["d"])))
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
    if op.startswith("recur"):
        B, T, D = case["B"], case["T"], case["D"]
        # decays of 0.9 to 0.999 a token where the gate is open: c softplus(lam) = -log decay
        m = -torch.log(uniform(D, lo=0.9, hi=0.999)) / DECAY
        s["lam"] = m + torch.log(-torch.expm1(-m))
        s["rg_bias"], s["ig_bias"] = normal(D, scale=0.1, of=torch.float32), normal(D, scale=0.1, of=torch.float32)
        if op == "recur_step":
            s["x"], s["rg"], s["ig"] = normal(B, D), normal(B, D), normal(B, D)
            s["z"] = normal(B, D) if case["gate"] else None
            s["h0"] = normal(B, D, scale=0.3, of=torch.float32)
            s["out_state"] = torch.empty_like(s["h0"])
            return s
        if case["packed"]:
            lens = _lengths(T, case["packed"], seed)
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            s["cu"], s["longest"], N = torch.tensor(cu, dtype=torch.int32, device=DEV), max(lens), len(lens)
        else:
            s["cu"], s["longest"], N = None, T, B
        s["x"] = normal(B, T, D)
        # both gates are halves of one projection, the output gate is the second half of the input's
        gates = normal(B, T, 2 * D)
        s["rg"], s["ig"] = gates[:, :, :D], gates[:, :, D:]
        s["z"] = normal(B, T, 2 * D)[:, :, D:] if case["gate"] else None
        s["h0"] = normal(N, D, scale=0.3, of=torch.float32) if case["state"] else None
        if op == "recur_train":
            s["dy"] = normal(B, T, D)
            s["dhT"] = normal(N, D, scale=0.3, of=torch.float32) if case["state"] else None
        return s
    if op.startswith("xent"):
        M, K, V = case["M"], case["K"], case["V"]
        s["x"], s["w"] = normal(M, K), normal(V, K, scale=1.5 * K ** -0.5)
        s["targets"] = torch.randint(0, V, (M,), generator=g, device=DEV)
        s["targets"][torch.rand(M, generator=g, device=DEV) < 0.05] = IGNORE  # padding
        if op == "xent_train":
            s["dloss"] = torch.full((M,), 1.0 / M, device=DEV)  # of the mean over the tokens
        return s
    B, T, d = case["B"], case["T"], case["d"]
    s["p"] = 0.1
    s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device=DEV)  # seed, number of the call
    s["x"] = normal(B, T, d)
    s["residual"] = normal(B, T, d, scale=3.0) if case["residual"] else None
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    # check_status=False, as a training or serving loop has it: reading the status word would wait for the GPU
    import chunkwise_delta_rule_02_gb300 as gdn
    op = s["op"]
    if op == "drop_fwd":
        return dict(y=gdn.dropout_forward(s["x"], s["p"], s["rng"], residual=s["residual"]))
    if op == "drop_bwd":
        return dict(dx=gdn.dropout_backward(s["x"], s["p"], s["rng"]))
    if op.startswith("xent"):
        loss, lse = gdn.xent_forward(s["x"], s["w"], s["targets"], ignore_index=IGNORE, check_status=False)
        if op == "xent_fwd":
            return dict(loss=loss, lse=lse)
        return dict(gdn.xent_backward(s["x"], s["w"], s["targets"], lse, s["dloss"], ignore_index=IGNORE, check_status=False), loss=loss, lse=lse)
    args = (s["x"], s["rg"], s["ig"], s["lam"])
    more = dict(rg_bias=s["rg_bias"], ig_bias=s["ig_bias"], z=s["z"], c=DECAY)
    if op == "recur_step":
        y, state = gdn.recur_step(*args, **more, state=s["h0"], out_state=s["out_state"])
        return dict(y=y, state=state)
    more.update(h0=s["h0"], cu_seqlens=s["cu"], check_status=False)
    if op == "recur_fwd":
        y, hT = gdn.recur_forward(*args, **more)
        return dict(y=y, state=hT)
    y, hT, saved = gdn.recur_forward(*args, **more, save=True)
    return dict(gdn.recur_backward(*args, **more, dy=s["dy"], dhT=s["dhT"], saved=saved), y=y, state=hT)


def _run_plain(s):
    return {"rec": _plain_recur, "xen": _plain_xent, "dro": _plain_drop}[s["op"][:3]](s)


def _dsilu(u):
    p = torch.sigmoid(u)
    return p * (1 + u * (1 - p))


def _doubling(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, in place, for sequences of at most `longest` tokens (a_t = 0 at their starts)."""
    k = 1
    while k < longest:
        b[k:] += a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _plain_recur(s):
    dt, D = s["x"].dtype, s["lam"].shape[0]
    silu = torch.nn.functional.silu
    flat = lambda v: v.reshape(-1, D).float()  # noqa: E731
    x, z = flat(s["x"]), None if s["z"] is None else flat(s["z"])
    r, i = torch.sigmoid(flat(s["rg"]) + s["rg_bias"]), torch.sigmoid(flat(s["ig"]) + s["ig_bias"])
    sp = torch.nn.functional.softplus(s["lam"])
    m = DECAY * sp * r
    decay, mag = torch.exp(-m), torch.sqrt(-torch.expm1(-2 * m))
    u = i * x
    if s["op"] == "recur_step":
        h = decay * s["h0"] + mag * u
        s["out_state"].copy_(h)
        return dict(y=(h if z is None else h * silu(z)).to(dt), state=s["out_state"])
    shape = s["x"].shape
    if s["cu"] is None:
        ends = (torch.arange(shape[0], device=DEV) + 1) * shape[1]
        starts = ends - shape[1]
    else:
        starts, ends = s["cu"][:-1].long(), s["cu"][1:].long()
    full = (ends > starts).nonzero()[:, 0]
    begin, end = starts[full], ends[full] - 1
    a, b = decay.clone(), mag * u
    a[begin] = 0
    if s["h0"] is not None:
        b[begin] += decay[begin] * s["h0"][full]
    h = _doubling(a, b, s["longest"])
    hT = torch.zeros(starts.numel(), D, device=DEV) if s["h0"] is None else s["h0"].clone()
    hT[full] = h[end]
    y = (h if z is None else h * silu(z)).to(dt).view(shape)
    if s["op"] == "recur_fwd":
        return dict(y=y, state=hT)
    dy = flat(s["dy"])
    dz = None if z is None else (dy * h * _dsilu(z)).to(dt).view(shape)
    dh = dy.clone() if z is None else dy * silu(z)
    # dh_t = dy_t + a_{t+1} dh_{t+1}: the same recurrence over the reversed axis
    a = torch.zeros_like(decay)
    a[:-1] = decay[1:]
    a[end] = 0
    if s["dhT"] is not None:
        dh[end] += s["dhT"][full]
    dh = _doubling(a.flip(0), dh.flip(0), s["longest"]).flip(0)
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[begin] = 0 if s["h0"] is None else s["h0"][full]
    q = m * dh * (u * decay.square() / mag - decay * before)
    drg = q * (1 - r)
    du = dh * mag
    dig = du * u * (1 - i)
    dh0 = None
    if s["h0"] is not None:
        dh0 = torch.zeros_like(s["h0"]) if s["dhT"] is None else s["dhT"].clone()
        dh0[full] = decay[begin] * dh[begin]
    out = lambda v: v.to(dt).view(shape)  # noqa: E731
    return dict(y=y, state=hT, dx=out(du * i), drg=out(drg), dig=out(dig), dz=dz, dlam=q.sum(0) * torch.sigmoid(s["lam"]) / sp,
                drg_bias=drg.sum(0), dig_bias=dig.sum(0), dh0=dh0)


def _plain_xent(s):
    x, w, t = s["x"].float(), s["w"].float(), s["targets"]
    logits = x @ w.t()
    valid = t != IGNORE
    at = torch.where(valid, t, 0)[:, None]
    top = logits.max(1, keepdim=True).values
    lse = (logits - top).exp().sum(1).log() + top[:, 0]
    loss = torch.where(valid, lse - logits.gather(1, at)[:, 0], 0.0)
    if s["op"] == "xent_fwd":
        return dict(loss=loss, lse=lse)
    g = torch.where(valid, s["dloss"], 0.0)
    d = logits.sub_(lse[:, None]).exp_().mul_(g[:, None])
    d.scatter_add_(1, at, -g[:, None])
    return dict(loss=loss, lse=lse, dx=(d @ w).to(s["x"].dtype), dw=(d.t() @ x).to(s["w"].dtype))


def _words(rng, n):
    """The generator's first n words: Philox 4x32 of 10 rounds, key = seed, counter = (index of a group of four, number of the call)."""
    low = 0xFFFFFFFF
    group = torch.arange((n + 3) // 4, device=DEV)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    c0, c1 = group & low, group >> 32
    c2, c3 = (rng[1] & low).expand_as(group), ((rng[1] >> 32) & low).expand_as(group)
    for _ in range(10):
        # 64-bit products of 32-bit numbers wrap in the sign only, so that their halves are right
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((q >> 32) & low) ^ c1 ^ k0, q & low, ((p >> 32) & low) ^ c3 ^ k1, p & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([c0, c1, c2, c3], 1).flatten()[:n]


def _plain_drop(s):
    x = s["x"].float()
    keep = (_words(s["rng"], x.numel()) >= round(s["p"] * 2 ** 32)).view(x.shape)
    y = torch.where(keep, x * (1 / (1 - s["p"])), 0.0)
    if s["op"] == "drop_bwd":
        return dict(dx=y.to(s["x"].dtype))
    return dict(y=(y if s["residual"] is None else s["residual"].float() + y).to(s["x"].dtype))


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    """What ``run`` returns, in float64: the recurrence token by token, the loss row block by row block, dropout word by word."""
    s = prepare(dict(case), seed)
    for k, v in s.items():
        if isinstance(v, torch.Tensor) and v.is_floating_point():
            s[k] = v.double()
    return {"rec": _exact_recur, "xen": _exact_xent, "dro": _exact_drop}[s["op"][:3]](s)


def _exact_recur(s):
    c, lam = s["case"], s["lam"]
    step = s["op"] == "recur_step"
    if step:
        for k in ("x", "rg", "ig", "z"):
            s[k] = s[k].unsqueeze(1) if s[k] is not None else None
    logistic = lambda v: 1 / (1 + torch.exp(-v))  # noqa: E731
    sp = torch.log1p(torch.exp(lam))
    r, i = logistic(s["rg"] + s["rg_bias"]), logistic(s["ig"] + s["ig_bias"])
    m = DECAY * sp * r
    a = torch.exp(-m)
    mag = (-torch.expm1(-2 * m)).sqrt()
    u = i * s["x"]
    B, T, D = u.shape
    cu = None if step else s["cu"]
    spans = [(b, 0, T, b) for b in range(B)] if cu is None else [(0, lo, hi, n) for n, (lo, hi) in enumerate(zip(cu[:-1].tolist(), cu[1:].tolist()))]
    h0 = torch.zeros(len(spans), D, dtype=torch.float64, device=DEV) if s["h0"] is None else s["h0"]
    first = {lo: n for _, lo, hi, n in spans if hi > lo}
    last = {hi - 1: n for _, lo, hi, n in spans if hi > lo}
    h, before = torch.empty_like(u), torch.empty_like(u)
    state, now = h0.clone(), h0
    for t in range(T):
        if cu is not None and t in first:
            now = h0[first[t]][None]
        before[:, t] = now
        now = a[:, t] * now + mag[:, t] * u[:, t]
        h[:, t] = now
        if cu is not None and t in last:
            state[last[t]] = now[0]
    if cu is None:
        state = now
    gate = None if s["z"] is None else logistic(s["z"])
    y = h if gate is None else h * s["z"] * gate
    if s["op"] != "recur_train":
        return dict(y=y[:, 0] if step else y, state=state)
    dz = None if gate is None else s["dy"] * h * (gate + s["z"] * gate * (1 - gate))
    g = s["dy"] if gate is None else s["dy"] * s["z"] * gate
    end = torch.zeros_like(h0) if s["dhT"] is None else s["dhT"]
    dh, dh0, back = torch.empty_like(u), end.clone(), end
    for t in reversed(range(T)):
        if cu is not None and t in last:
            back = end[last[t]][None]
        dh[:, t] = back + g[:, t]
        back = a[:, t] * dh[:, t]
        if cu is not None and t in first:
            dh0[first[t]] = back[0]
    if cu is None:
        dh0 = back
    dlog = a * dh * (before - u * a / mag)           # gradient of log a = -m
    dr = -DECAY * sp * dlog
    drg, dig = dr * r * (1 - r), dh * mag * s["x"] * i * (1 - i)
    rows = lambda v: v.sum((0, 1))  # noqa: E731
    return dict(y=y, state=state, dx=dh * mag * i, drg=drg, dig=dig, dz=dz, dlam=rows(-DECAY * r * dlog) * logistic(lam),
                drg_bias=rows(drg), dig_bias=rows(dig), dh0=dh0 if s["h0"] is not None else None)


def _exact_xent(s):
    x, w, t = s["x"], s["w"], s["targets"]
    train = s["op"] == "xent_train"
    loss, lse = torch.empty(x.shape[0], dtype=torch.float64, device=DEV), torch.empty(x.shape[0], dtype=torch.float64, device=DEV)
    dx, dw = (torch.empty_like(x), torch.zeros_like(w)) if train else (None, None)
    for lo in range(0, x.shape[0], 2048):
        part = slice(lo, lo + 2048)
        logits = torch.einsum("mk,vk->mv", x[part], w)
        lse[part] = torch.logsumexp(logits, 1)
        counted = (t[part] != IGNORE).double()
        rows = torch.arange(logits.shape[0], device=DEV)
        target = t[part].clamp(min=0)
        loss[part] = counted * (lse[part] - logits[rows, target])
        if train:
            p = torch.softmax(logits, 1)
            p[rows, target] -= 1
            p *= (counted * s["dloss"][part])[:, None]
            dx[part] = torch.einsum("mv,vk->mk", p, w)
            dw += torch.einsum("mv,mk->vk", p, x[part])
    return dict(loss=loss, lse=lse, dx=dx, dw=dw) if train else dict(loss=loss, lse=lse)


def _exact_drop(s):
    """The generator on 16-bit halves, apart from the plain form's 64-bit products."""
    half = 0xFFFF
    seed, call = (int(v) for v in s["rng"].tolist())
    n = s["x"].numel()
    group = torch.arange((n + 3) // 4, device=DEV)

    def product(c, k):
        """(high, low) 32 bits of c times the constant k."""
        cl, ch, kl, kh = c & half, c >> 16, k & half, k >> 16
        mid = cl * kh + ((cl * kl) >> 16)
        mid2 = ch * kl + (mid & half)
        return ch * kh + (mid >> 16) + (mid2 >> 16), ((mid2 & half) << 16) | ((cl * kl) & half)

    word = lambda v, shift: torch.full_like(group, (v >> shift) & 0xFFFFFFFF)  # noqa: E731
    c = [group % 2 ** 32, group // 2 ** 32, word(call, 0), word(call, 32)]
    for j in range(10):
        keys = ((seed & 0xFFFFFFFF) + j * 0x9E3779B9) % 2 ** 32, ((seed >> 32) + j * 0xBB67AE85) % 2 ** 32
        high0, low0 = product(c[0], 0xD2511F53)
        high1, low1 = product(c[2], 0xCD9E8D57)
        c = [high1 ^ c[1] ^ keys[0], low1, high0 ^ c[3] ^ keys[1], low0]
    words = torch.stack(c, -1).reshape(-1)[:n].view(s["x"].shape)
    y = s["x"] * (words.double() / 2 ** 32 >= round(s["p"] * 2 ** 32) / 2 ** 32) / (1 - s["p"])
    if s["op"] == "drop_bwd":
        return dict(dx=y)
    return dict(y=y if s["residual"] is None else s["residual"] + y)


# ------------------------------------------------------------------ work


def work(case):
    op, e = case["op"], 2 if case["type"] == "bf16" else 4
    if op.startswith("xent"):
        M, K, V = case["M"], case["K"], case["V"]
        once = (M + V) * K * e + M * 16  # x and w; targets, loss, lse
        if op == "xent_fwd":
            return dict(bytes=once, flops=2 * M * V * K + 4 * M * V)
        return dict(bytes=2 * once, flops=6 * M * V * K + 8 * M * V)
    if op.startswith("drop"):
        n = case["B"] * case["T"] * case["d"]
        return dict(bytes=n * e * (3 if case["residual"] else 2), flops=n * 12)
    n, D, z = case["B"] * case["T"] * case["D"], case["D"], 1 if case["gate"] else 0
    st = (case["packed"] or case["B"]) * D * 4
    if op == "recur_train":  # x, both gates, dy in; y, their gradients out; the output gate and its gradient
        return dict(bytes=n * e * (8 + 2 * z) + st * (4 if case["state"] else 1) + 24 * D, flops=n * (60 + 15 * z))
    return dict(bytes=n * e * (4 + z) + st * (2 if case["state"] else 1) + 12 * D, flops=n * (25 + 5 * z))
