"""A small hybrid language model on the package's operators: gated delta rule blocks and selective state
space blocks, trained on a synthetic copy task and then decoded token by token.

Each block is a residual norm (the sum of the stream and the block before it, its scale and the norm in one
pass), projections, short causal convolutions, the delta rule or the scan, a gated norm (delta rule) or the
scan's own gate, and an output projection.  The convolutions read the token-major projections and write what
the delta rule reads; the gated norm reads that layout and writes the projection's: the forward pass has no
transposition or copy in between (gradients come back in the axes' order, contiguous).  Decoding keeps, per block, the last taps of the convolutions and the recurrent states.

    python examples/hybrid_blocks.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunkwise_delta_rule_02_gb300 as gdn  # noqa: E402

BF = torch.bfloat16


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias):
        ctx.save_for_backward(x, w, bias)
        return gdn.conv_forward(x, w, bias, want_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        x, w, bias = ctx.saved_tensors
        g = gdn.conv_backward(x, w, bias, None, dy)
        return g["dx"], g["dw"], g["dbias"]


class DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, beta, gate):
        ctx.save_for_backward(q, k, v, beta, gate)
        return gdn.forward(q, k, v, beta, gate, want_state=False, check_status=False)[0]

    @staticmethod
    def backward(ctx, dO):
        q, k, v, beta, gate = ctx.saved_tensors
        g = gdn.backward(q, k, v, beta, gate, None, dO.contiguous(), None, check_status=False)
        return g["dq"], g["dk"], g["dv"], g["dbeta"], g["dg"]


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias):
        y, _, saved = gdn.scan_forward(x, dt, A, B, C, D, z, dt_bias, want_state=False, save=True)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, saved)
        return y

    @staticmethod
    def backward(ctx, dy):
        *args, saved = ctx.saved_tensors
        g = gdn.scan_backward(*args, dy=dy.contiguous(), saved=saved)
        return tuple(g[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias"))


class GatedNorm(torch.autograd.Function):
    """rms(o) w silu(z) of head-major o and token-major z (as a [B,H,T,d] view), token-major out."""

    @staticmethod
    def forward(ctx, o, w, z):
        ctx.save_for_backward(o, w, z)
        B, H, T, d = o.shape
        out = torch.empty(B, T, H, d, dtype=o.dtype, device=o.device).transpose(1, 2)
        return gdn.norm_forward(o, w, z=z, out=out)

    @staticmethod
    def backward(ctx, dy):
        o, w, z = ctx.saved_tensors
        g = gdn.norm_backward(o, w, dy, z=z)
        return g["dx"], g["dw"], g["dz"]


class ResidualNorm(torch.autograd.Function):
    """(rms(r) w, r) with r = residual + scale * x."""

    @staticmethod
    def forward(ctx, x, residual, w, scale):
        y, r = gdn.norm_forward(x, w, residual=residual, res_scale=scale)
        ctx.save_for_backward(x, w, scale, r)
        return y, r

    @staticmethod
    def backward(ctx, dy, dr):
        x, w, scale, r = ctx.saved_tensors
        g = gdn.norm_backward(x, w, dy.contiguous(), sum=r, dsum=dr.contiguous(), res_scale=scale)
        return g["dx"], g["dresidual"], g["dw"], g["dres_scale"]


class DeltaBlock(torch.nn.Module):
    """Gated delta rule: q, k, v through a convolution each, a gated norm per head behind it."""

    def __init__(self, width, heads, d, taps=4):
        super().__init__()
        self.heads, self.d, self.C = heads, d, heads * d
        p = lambda *s, scale: torch.nn.Parameter(torch.randn(*s) * scale)  # noqa: E731
        self.proj = p(width, 4 * self.C, scale=width ** -0.5)       # q, k, v, z
        self.steps = p(width, 2 * heads, scale=width ** -0.5)       # beta, gate
        self.taps = torch.nn.ParameterList([p(self.C, taps, scale=taps ** -0.5) for _ in range(3)])
        self.tap_bias = torch.nn.ParameterList([torch.nn.Parameter(torch.zeros(self.C)) for _ in range(3)])
        self.norm = torch.nn.Parameter(torch.ones(d))
        self.out = p(self.C, width, scale=self.C ** -0.5)

    def _projected(self, u):
        qkvz = u @ self.proj.to(BF)
        bg = (u @ self.steps.to(BF)).float()
        return qkvz.split(self.C, -1), torch.sigmoid(bg[..., :self.heads]), -torch.nn.functional.softplus(bg[..., self.heads:])

    def forward(self, u):
        (*qkv, z), beta, gate = self._projected(u)
        by_head = lambda t: t.unflatten(-1, (self.heads, self.d)).transpose(1, 2)  # noqa: E731
        q, k, v = (Conv.apply(by_head(t), w, b) for t, w, b in zip(qkv, self.taps, self.tap_bias))
        o = DeltaRule.apply(q, k, v, beta.transpose(1, 2).to(BF).contiguous(), gate.transpose(1, 2).contiguous())
        return GatedNorm.apply(o, self.norm, by_head(z)).transpose(1, 2).flatten(2) @ self.out.to(BF)

    def start(self, n, device):
        return dict(taps=[torch.zeros(n, w.shape[1] - 1, self.C, dtype=BF, device=device) for w in self.taps],
                    state=torch.zeros(n, self.heads, self.d, self.d, device=device))

    def step(self, u, s):
        (*qkv, z), beta, gate = self._projected(u)
        by_head = lambda t: t.unflatten(-1, (self.heads, self.d))  # noqa: E731
        q, k, v = (by_head(gdn.conv_step(t, w, b, st, out_state=st)[0])
                   for t, w, b, st in zip(qkv, self.taps, self.tap_bias, s["taps"]))
        o, _ = gdn.decode_step(q, k, v, beta.to(BF).contiguous(), gate.contiguous(), state=s["state"], out_state=s["state"])
        return gdn.norm_forward(o, self.norm, z=by_head(z)).flatten(1) @ self.out.to(BF)


class ScanBlock(torch.nn.Module):
    """Selective state space block: one convolution, steps and B, C from its output, the gate in the scan."""

    def __init__(self, width, channels, states, low=16, taps=4):
        super().__init__()
        self.channels, self.states, self.low = channels, states, low
        p = lambda *s, scale: torch.nn.Parameter(torch.randn(*s) * scale)  # noqa: E731
        self.proj = p(width, 2 * channels, scale=width ** -0.5)     # x, z
        self.taps, self.tap_bias = p(channels, taps, scale=taps ** -0.5), torch.nn.Parameter(torch.zeros(channels))
        self.select = p(channels, low + 2 * states, scale=channels ** -0.5)
        self.widen = p(low, channels, scale=low ** -0.5)
        self.log_A = torch.nn.Parameter(torch.log(torch.arange(1, states + 1).float()).repeat(channels, 1))
        self.skip = torch.nn.Parameter(torch.ones(channels))
        step = torch.exp(torch.rand(channels) * math.log(100.0) + math.log(1e-3))
        self.dt_bias = torch.nn.Parameter(step + torch.log(-torch.expm1(-step)))
        self.out = p(channels, width, scale=channels ** -0.5)

    def _selected(self, x):
        s = x @ self.select.to(BF)
        return s[..., :self.low] @ self.widen.to(BF), s[..., self.low:self.low + self.states], s[..., self.low + self.states:]

    def forward(self, u):
        x, z = (u @ self.proj.to(BF)).split(self.channels, -1)
        x = Conv.apply(x, self.taps, self.tap_bias)
        dt, B, C = self._selected(x)
        return Scan.apply(x, dt, -torch.exp(self.log_A), B, C, self.skip, z, self.dt_bias) @ self.out.to(BF)

    def start(self, n, device):
        return dict(taps=torch.zeros(n, self.taps.shape[1] - 1, self.channels, dtype=BF, device=device),
                    state=torch.zeros(n, self.channels, self.states, device=device))

    def step(self, u, s):
        x, z = (u @ self.proj.to(BF)).split(self.channels, -1)
        x, _ = gdn.conv_step(x, self.taps, self.tap_bias, s["taps"], out_state=s["taps"])
        dt, B, C = self._selected(x)
        y, _ = gdn.scan_step(x, dt, -torch.exp(self.log_A), B, C, self.skip, z, self.dt_bias, s["state"], out_state=s["state"])
        return y @ self.out.to(BF)


class HybridModel(torch.nn.Module):
    def __init__(self, vocab=64, width=256, heads=2, d=128, channels=512, states=16, pairs=1):
        super().__init__()
        self.embed = torch.nn.Parameter(torch.randn(vocab, width) * 0.5)
        blocks = []
        for _ in range(pairs):
            blocks += [DeltaBlock(width, heads, d), ScanBlock(width, channels, states)]
        self.blocks = torch.nn.ModuleList(blocks)
        self.norms = torch.nn.ParameterList([torch.nn.Parameter(torch.ones(width)) for _ in range(len(blocks) + 1)])
        self.scales = torch.nn.ParameterList([torch.nn.Parameter(torch.ones(width)) for _ in range(len(blocks) + 1)])

    def forward(self, tokens):
        r = self.embed[tokens].to(BF)
        x = torch.zeros_like(r)
        for i, block in enumerate(self.blocks):
            u, r = ResidualNorm.apply(x, r, self.norms[i], self.scales[i])
            x = block(u)
        u, _ = ResidualNorm.apply(x, r, self.norms[-1], self.scales[-1])
        return u @ self.embed.t().to(BF)

    def start(self, n):
        return [b.start(n, self.embed.device) for b in self.blocks]

    @torch.no_grad()
    def step(self, tokens, states):
        """Logits of the next token for tokens [n]; the states move on in place."""
        r = self.embed[tokens].to(BF)
        x = torch.zeros_like(r)
        for i, (block, s) in enumerate(zip(self.blocks, states)):
            u, r = gdn.norm_forward(x, self.norms[i], residual=r, res_scale=self.scales[i])
            x = block.step(u, s)
        u, _ = gdn.norm_forward(x, self.norms[-1], residual=r, res_scale=self.scales[-1])
        return u @ self.embed.t().to(BF)


def batch(n, T, vocab, gen):
    """Sequences that repeat a random span of theirs: the second half is predictable from the first."""
    span = torch.randint(0, vocab, (n, T // 2), generator=gen)
    return torch.cat([span, span], 1).cuda()


def train(model, steps=30, n=8, T=128, vocab=64, seed=0):
    """The losses of `steps` training steps."""
    gen = torch.Generator().manual_seed(seed)
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        tokens = batch(n, T, vocab, gen)
        logits = model(tokens[:, :-1]).float()
        loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), tokens[:, 1:].flatten())
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def main():
    torch.manual_seed(0)
    model = HybridModel().cuda()
    losses = train(model)
    print("loss %.3f -> %.3f" % (losses[0], losses[-1]))
    tokens = batch(4, 64, 64, torch.Generator().manual_seed(1))
    with torch.no_grad():
        whole = model(tokens).float()
    states = model.start(4)
    single = torch.stack([model.step(tokens[:, t], states).float() for t in range(tokens.shape[1])], 1)
    print("token by token against the whole sequence: %.4f" % float((single - whole).norm() / whole.norm()))


if __name__ == "__main__":
    main()
