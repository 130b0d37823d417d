"""A hybrid token mixer: half of the channels through a gated long convolution,
half through the gated delta rule.

    python examples/hybrid_mixer.py [--batch B] [--tokens T] [--steps N]

The block normalises its input, projects it, and mixes along the sequence twice:
a Hyena-style branch w_out . conv(u . w_in, k) and a delta-rule branch whose
queries and keys are normed for each head and rotated by position.  The script
trains the delta-rule branch's projections for a few steps (forward, gradients,
update), then runs a prompt and decodes tokens one by one from the states that
the prompt left, checking them against the prompt run as a whole.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fft_long_convolution_gb300 as F  # noqa: E402


class HybridMixer:
    """hidden channels: hidden/2 by the convolution, hidden/2 as heads of 64 by
    the delta rule."""

    def __init__(self, hidden: int, tokens: int, dtype=torch.bfloat16, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*s):
            return torch.randn(*s, generator=gen, device="cuda")

        self.dtype, self.half, self.D = dtype, hidden // 2, 64
        self.heads = self.half // self.D
        # the convolution: u, w_in and w_out from one projection, one decaying kernel per channel
        self.conv = F.Plan(tokens, dtype)
        self.w_conv = (randn(hidden, 3 * self.half) * hidden ** -0.5).to(dtype)
        decay = torch.exp(-torch.linspace(1, 8, self.half, device="cuda")[:, None] * torch.arange(tokens, device="cuda") / tokens)
        self.k_f = self.conv.kernel_fft((randn(self.half, tokens) * decay * tokens ** -0.5).contiguous())
        # the delta rule: queries, keys and values from one projection, gates from another
        self.rule = F.DeltaRule(self.D, self.D, dtype)
        self.norm = F.QKNorm(self.D, dtype, norm="l2", rotary=self.D // 2)
        self.w_qkv = (randn(hidden, 3 * self.half) * hidden ** -0.5).to(dtype)
        self.w_gate = (randn(hidden, 2 * self.heads) * hidden ** -0.5).to(dtype)
        self.wq, self.wk = torch.ones(self.D, device="cuda"), torch.ones(self.D, device="cuda")
        angle = torch.arange(tokens, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, self.D // 4, device="cuda") / (self.D // 4))
        self.cos, self.sin = angle.cos().contiguous(), angle.sin().contiguous()

    def convolution(self, x):
        """x [B, N, hidden] -> [B, N, hidden/2]; the plan works on [B, H, N]."""
        u, w_in, w_out = (x @ self.w_conv).transpose(1, 2).contiguous().split(self.half, 1)
        return self.conv.forward_gated(u.contiguous(), w_in.contiguous(), w_out.contiguous(), self.k_f).transpose(1, 2)

    def projections(self, x):
        """q, k, v as views of one projection, log decays and betas."""
        q, k, v = ((x @ self.w_qkv)[..., i * self.half:(i + 1) * self.half].unflatten(2, (self.heads, self.D)) for i in range(3))
        a, b = (x @ self.w_gate).float().split(self.heads, 2)
        return q, k, v, (-torch.nn.functional.softplus(a - 3.0)).to(self.dtype), torch.sigmoid(b).to(self.dtype)

    def normed(self, q, k, positions=None):
        return self.norm.forward(q, k, wq=self.wq, wk=self.wk, cos=self.cos, sin=self.sin, positions=positions)

    def prompt(self, x, state=None, positions=None):
        q, k, v, g, beta = self.projections(x)
        q, k = self.normed(q, k, positions)
        return self.rule.forward(q, k, v, g, beta, state=state)

    def decode(self, x, state, position):
        """One token a row, [B, 1, hidden], against the states (updated in place)."""
        q, k, v, g, beta = self.projections(x)
        q, k = self.normed(q, k, torch.full(x.shape[:2], position, dtype=torch.int32, device=x.device))
        return self.rule.step(q, k, v, g, beta, state)

    def train_step(self, x, target, lr):
        """One step on w_qkv, lr of its norm long: the delta-rule branch against target."""
        q, k, v, g, beta = self.projections(x)
        qn, kn = self.normed(q, k)
        o, _, saved = self.rule.forward(qn, kn, v, g, beta, save=True)
        miss = o.float() - target.float()
        do = (2.0 / miss.numel() * miss * 1024.0).to(self.dtype)  # loss scaled by 1024 for 16 bits
        dqn, dkn, dv, _, _, _ = self.rule.backward(do, qn, kn, v, g, beta, saved)
        dq, dk, _, _ = self.norm.backward(dqn, dkn, q, k, wq=self.wq, wk=self.wk, cos=self.cos, sin=self.sin)
        d = torch.cat([t.flatten(2) for t in (dq, dk, dv)], 2)
        grad = (x.flatten(0, 1).t() @ d.flatten(0, 1)).float()
        w = self.w_qkv.float()
        self.w_qkv = (w - lr * w.norm() / grad.norm() * grad).to(self.dtype)
        return float(miss.square().mean())


def run(batch: int = 2, tokens: int = 4096, steps: int = 5, hidden: int = 768, decode: int = 8) -> dict:
    net = HybridMixer(hidden, tokens)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(batch, tokens, hidden, generator=gen, device="cuda").to(net.dtype)
    target = HybridMixer(hidden, tokens, seed=2).prompt(x)[0]  # what another block's branch answers
    losses = [net.train_step(x, target, lr=0.05) for _ in range(steps)]
    # the whole block on a prompt
    o, state = net.prompt(x[:, :tokens - decode])
    y = torch.cat([net.convolution(x), net.prompt(x)[0].flatten(2)], 2)
    # the rest token by token
    last = [net.decode(x[:, t:t + 1], state, t) for t in range(tokens - decode, tokens)]
    whole = net.prompt(x)[0][:, tokens - decode:]
    diff = (torch.cat(last, 1).float() - whole.float()).norm() / whole.float().norm()
    assert net.rule.device_status() == 0 and net.conv.device_status() == 0
    return {"losses": losses, "shape": tuple(y.shape), "decode_difference": float(diff)}


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    r = run(a.batch, a.tokens, a.steps)
    print("loss", " -> ".join(f"{x:.5f}" for x in r["losses"]))
    print("block output", r["shape"], "decoded tokens against the whole prompt:", f"{r['decode_difference']:.1e}")
