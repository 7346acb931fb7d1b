"""A recurrent sequence block built on the library: short causal convolution,
selective scan and gated group norm between two projections.

    python examples/sequence_block.py        # on an MI355X

trains a small model of such blocks on a synthetic task (repeat what was seen a
fixed number of tokens ago), then reads a batch of prompts of unequal lengths in
one pass and continues each token by token from the carried states, and checks
that the steps give what one pass over the whole sequence gives.
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_recurrence_scans_amd as lrs  # noqa: E402


class CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias):
        ctx.save_for_backward(x, w, bias)
        return lrs.mi_causal_conv_fwd(x, w, bias, act="silu")[0]

    @staticmethod
    def backward(ctx, dy):
        x, w, bias = ctx.saved_tensors
        return lrs.mi_causal_conv_bwd(x, w, bias, None, dy, act="silu")[:3]


class SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, delta, A, Bm, Cm, skip, delta_bias):
        y, _, states = lrs.mi_selective_scan_fwd(u, delta, A, Bm, Cm, skip, None, delta_bias, save_states=True)
        ctx.save_for_backward(u, delta, A, Bm, Cm, skip, delta_bias, states)
        return y

    @staticmethod
    def backward(ctx, dy):
        u, delta, A, Bm, Cm, skip, delta_bias, states = ctx.saved_tensors
        g = lrs.mi_selective_scan_bwd(u, delta, A, Bm, Cm, states, dy, None, skip, None, delta_bias)
        return g[0], g[1], g[2], g[3], g[4], g[5], g[7]


class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, z, groups):
        ctx.save_for_backward(x, w, z)
        ctx.groups = groups
        return lrs.mi_group_norm_fwd(x, w, None, z, groups=groups, centered=False)

    @staticmethod
    def backward(ctx, dy):
        x, w, z = ctx.saved_tensors
        dx, dw, _, dz = lrs.mi_group_norm_bwd(x, w, None, dy, z, groups=ctx.groups, centered=False)
        return dx, dw, dz, None


class Block(torch.nn.Module):
    """x + out(norm(scan(conv(in(x)))) gated)."""

    def __init__(self, width, inner, states=16, taps=4, rank=8, groups=4):
        super().__init__()
        self.inner, self.states, self.taps, self.rank, self.groups = inner, states, taps, rank, groups
        self.inp = torch.nn.Linear(width, 2 * inner, bias=False)
        self.conv_w = torch.nn.Parameter(torch.randn(inner, taps) * taps ** -0.5)
        self.conv_b = torch.nn.Parameter(torch.zeros(inner))
        self.proj = torch.nn.Linear(inner, rank + 2 * states, bias=False)
        self.rate = torch.nn.Linear(rank, inner, bias=False)
        target = torch.exp(torch.empty(inner).uniform_(-6.9, -2.3))  # rates of 1e-3 to 1e-1
        self.rate_b = torch.nn.Parameter(target + torch.log(-torch.expm1(-target)))
        self.log_A = torch.nn.Parameter(torch.log(torch.arange(1, states + 1).float()).repeat(inner, 1))
        self.skip = torch.nn.Parameter(torch.ones(inner))
        self.norm_w = torch.nn.Parameter(torch.ones(inner))
        self.out = torch.nn.Linear(inner, width, bias=False)

    def _gates(self, v):
        r, Bm, Cm = self.proj(v).split([self.rank, self.states, self.states], -1)
        return self.rate(r), Bm.unsqueeze(-2), Cm.unsqueeze(-2), -torch.exp(self.log_A)

    def forward(self, x):
        v, z = self.inp(x).chunk(2, -1)
        v = CausalConv.apply(v, self.conv_w, self.conv_b)
        delta, Bm, Cm, A = self._gates(v)
        y = SelectiveScan.apply(v, delta, A, Bm, Cm, self.skip, self.rate_b)
        return x + self.out(GatedNorm.apply(y, self.norm_w, z, self.groups))

    @torch.no_grad()
    def prompt(self, x, lengths):
        """(y, state) of a batch of prompts of the given lengths."""
        v, z = self.inp(x).chunk(2, -1)
        v, taps = lrs.mi_causal_conv_fwd(v, self.conv_w, self.conv_b, act="silu", lengths=lengths)
        delta, Bm, Cm, A = self._gates(v)
        y, h, _ = lrs.mi_selective_scan_fwd(v, delta, A, Bm, Cm, self.skip, None, self.rate_b, lengths=lengths)
        y = lrs.mi_group_norm_fwd(y, self.norm_w, None, z, groups=self.groups, centered=False)
        return x + self.out(y), (taps, h)

    @torch.no_grad()
    def step(self, x, state):
        """One token for every sequence; the state is updated in place."""
        taps, h = state
        v, z = self.inp(x).chunk(2, -1)
        v, _ = lrs.mi_causal_conv_step(v, self.conv_w, self.conv_b, taps, act="silu", x_out=taps)
        delta, Bm, Cm, A = self._gates(v)
        y, _ = lrs.mi_selective_scan_step(v, delta, A, Bm, Cm, h, self.skip, None, self.rate_b, h_out=h)
        y = lrs.mi_group_norm_fwd(y, self.norm_w, None, z, groups=self.groups, centered=False)
        return x + self.out(y)


class Model(torch.nn.Module):
    def __init__(self, vocab=16, width=64, inner=128, depth=2):
        super().__init__()
        self.embed = torch.nn.Embedding(vocab, width)
        self.blocks = torch.nn.ModuleList(Block(width, inner) for _ in range(depth))
        self.head = torch.nn.Linear(width, vocab)

    def forward(self, tokens):
        x = self.embed(tokens)
        for b in self.blocks:
            x = b(x)
        return self.head(x)

    @torch.no_grad()
    def prompt(self, tokens, lengths):
        x, states = self.embed(tokens), []
        for b in self.blocks:
            x, st = b.prompt(x, lengths)
            states.append(st)
        return self.head(x), states

    @torch.no_grad()
    def step(self, tokens, states):
        x = self.embed(tokens)
        for b, st in zip(self.blocks, states):
            x = b.step(x, st)
        return self.head(x)


def train(model, steps, lag=3, batch=16, length=64, vocab=16):
    """Predict the token seen `lag` steps ago; the losses of every step."""
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    g = torch.Generator("cuda").manual_seed(1)
    losses = []
    for _ in range(steps):
        tokens = torch.randint(0, vocab, (batch, length), device="cuda", generator=g)
        loss = F.cross_entropy(model(tokens)[:, lag:].reshape(-1, vocab), tokens[:, :-lag].reshape(-1))
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return [float(x) for x in losses]


@torch.no_grad()
def serve(model, lengths, extra, vocab=16):
    """Largest difference between stepping from carried states and one pass."""
    B, T = len(lengths), max(lengths)
    g = torch.Generator("cuda").manual_seed(2)
    whole = torch.randint(0, vocab, (B, T + extra), device="cuda", generator=g)
    want = model(whole)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    logits, states = model.prompt(whole[:, :T], n)
    rows = torch.arange(B, device="cuda")
    worst = max(float((logits[b, :k] - want[b, :k]).abs().max()) for b, k in enumerate(lengths) if k)
    for i in range(extra):
        at = n.long() + i
        got = model.step(whole[rows, at], states)
        worst = max(worst, float((got - want[rows, at]).abs().max()))
    return worst


def main():
    torch.manual_seed(0)
    model = Model().cuda()
    losses = train(model, 200)
    print("loss %.3f -> %.3f over %d steps" % (losses[0], losses[-1], len(losses)))
    print("steps against one pass: largest logit difference %.2e" % serve(model, [40, 17, 0, 33], 12))


if __name__ == "__main__":
    main()
