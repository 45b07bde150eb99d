"""Plain 64-bit forms of the gated linear recurrence and of dropout, on the CPU, for the tests: token by token and
word by word; gradients by differentiating them."""
import torch

import layers_ref

F64 = torch.float64


def recur(x, rg, ig, lam, rg_bias=None, ig_bias=None, z=None, h0=None, c=8.0, cu=None):
    """x [B,T,D] -> (y, hT)."""
    B, T, D = x.shape
    r = torch.sigmoid(rg if rg_bias is None else rg + rg_bias)
    i = torch.sigmoid(ig if ig_bias is None else ig + ig_bias)
    m = c * torch.nn.functional.softplus(lam) * r
    a, s = torch.exp(-m), torch.sqrt(-torch.expm1(-2 * m))
    rows, ends = [], []
    for b, lo, hi, n in layers_ref.spans(B, T, cu):
        h = torch.zeros(D, dtype=x.dtype) if h0 is None else h0[n]
        for t in range(lo, hi):
            h = a[b, t] * h + s[b, t] * i[b, t] * x[b, t]
            rows.append(h)
        ends.append(h)
    h = torch.stack(rows).reshape(B, T, D) if rows else x.clone()
    hT = torch.stack(ends) if ends else torch.zeros(0, D, dtype=x.dtype)
    return (h if z is None else h * z * torch.sigmoid(z)), hT


def words(seed, call, n):
    """The first n words of Philox 4x32 of 10 rounds (Salmon et al. 2011), in Python's integers."""
    low = (1 << 32) - 1
    out = []
    for group in range((n + 3) // 4):
        c = [group & low, group >> 32, call & low, (call >> 32) & low]
        k0, k1 = seed & low, (seed >> 32) & low
        for _ in range(10):
            p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(q >> 32) ^ c[1] ^ k0, q & low, (p >> 32) ^ c[3] ^ k1, p & low]
            k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
        out += c
    return out[:n]


def keep(seed, call, p, shape):
    n = 1
    for v in shape:
        n *= v
    return (torch.tensor(words(seed, call, n), dtype=torch.int64) >= int(p * 2 ** 32 + 0.5)).view(shape)


def dropout(x, p, seed, call, residual=None):
    y = torch.where(keep(seed, call, p, x.shape), x / (1 - p), torch.zeros((), dtype=x.dtype))
    return y if residual is None else residual + y
