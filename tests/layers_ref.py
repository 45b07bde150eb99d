"""Plain 64-bit forms of the layer operators, on the CPU, for the tests: token by token or sequence by
sequence, gradients by differentiating these forms."""
import torch

F64 = torch.float64


def spans(B, T, cu):
    """(batch row, first token, end, sequence)."""
    if cu is None:
        return [(b, 0, T, b) for b in range(B)]
    cu = [int(v) for v in cu]
    return [(0, cu[i], cu[i + 1], i) for i in range(len(cu) - 1)]


def silu(u):
    return u * torch.sigmoid(u)


def conv(x, w, bias, s0, cu=None, act=True):
    """x [B,H,T,d] -> (y, sT); s0 [N,W-1,C] or None."""
    B, H, T, d = x.shape
    C, W = w.shape
    sp = spans(B, T, cu)
    ys, ends = [], []
    for b, lo, hi, n in sp:
        first = torch.zeros(W - 1, C, dtype=x.dtype) if s0 is None else s0[n]
        rows = torch.cat([first, x[b, :, lo:hi].permute(1, 0, 2).reshape(hi - lo, C)])
        if hi > lo:
            pre = torch.stack([(rows[t:t + W] * w.t()).sum(0) for t in range(hi - lo)])
            if bias is not None:
                pre = pre + bias
            ys.append(silu(pre) if act else pre)
        ends.append(rows[hi - lo:])
    y = torch.cat(ys).reshape(B, T, H, d).permute(0, 2, 1, 3) if ys else x.clone()
    sT = torch.stack(ends) if ends else torch.zeros(0, W - 1, C, dtype=x.dtype)
    return y, sT


def scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, cu=None, softplus=True):
    """x, dt, z [B,T,D]; Bm, Cm [B,T,G,N] -> (y, hT)."""
    B, T, Dc = x.shape
    G, N = Bm.shape[2:]
    raw = dt if dt_bias is None else dt + dt_bias
    delta = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())) if softplus else raw
    wide = lambda v: v.repeat_interleave(Dc // G, 0)  # noqa: E731
    rows, ends = [], []
    for b, lo, hi, n in spans(B, T, cu):
        h = torch.zeros(Dc, N, dtype=x.dtype) if h0 is None else h0[n]
        for t in range(lo, hi):
            u = delta[b, t][:, None]
            h = torch.exp(u * A) * h + u * x[b, t][:, None] * wide(Bm[b, t])
            rows.append((h * wide(Cm[b, t])).sum(-1))
        ends.append(h)
    o = torch.stack(rows).reshape(B, T, Dc) if rows else torch.zeros_like(x)
    if D is not None:
        o = o + D * x
    y = o if z is None else o * silu(z)
    return y, torch.stack(ends) if ends else torch.zeros(0, Dc, N, dtype=x.dtype)


def norm(x, w, z=None, residual=None, res_scale=None, eps=1e-6):
    """x [B,H,T,d]; w [d] or [H,d] -> (y, r)."""
    r = x
    if residual is not None:
        r = residual + (x if res_scale is None else res_scale * x)
    y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * (w if w.dim() == 1 else w[:, None])
    return (y if z is None else y * silu(z)), r


def grads(outs, ups, leaves):
    """Gradients of sum <out, up> for every leaf (zeros where it has no part)."""
    loss = sum((o * u).sum() for o, u in zip(outs, ups) if u is not None)
    if not torch.is_tensor(loss) or not loss.requires_grad:
        return [torch.zeros_like(v) for v in leaves]
    got = torch.autograd.grad(loss, leaves, allow_unused=True)
    return [torch.zeros_like(v) if g is None else g for v, g in zip(leaves, got)]


def leaf(t):
    return None if t is None else t.detach().cpu().to(F64).requires_grad_(True)


def d64(t):
    return None if t is None else t.detach().cpu().to(F64)


def err(a, ref):
    """Relative Frobenius error (absolute where the reference is zero)."""
    a, ref = a.detach().cpu().to(F64), ref.detach().to(F64)
    assert a.shape == ref.shape, (a.shape, ref.shape)
    n = float(ref.norm())
    return float((a - ref).norm()) / n if n else float(a.norm())
