"""A Mamba-2 mixer trained and served with the packed-token operators.

    python examples/mamba2_mixer.py

Training: documents of several lengths in one packed batch go through the
input projection, causal_conv1d_varlen_fwd, ssd_varlen_fwd (which keeps every
chunk's state in 8 bits), the gate and the output projection, and back through
ssd_varlen_bwd and causal_conv1d_varlen_bwd.  Serving: prompts of several
lengths fill the requests' caches in one call, and conv1d_ssd_update adds a
token to each of them.  Random weights and data.
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from state_space_model_scan_amd import (causal_conv1d_varlen_bwd, causal_conv1d_varlen_fwd,  # noqa: E402
                                        conv1d_ssd_update, ssd_checkpoint_slots, ssd_varlen_bwd, ssd_varlen_fwd)

HEADDIM = 64


class Mixer:
    """Weights in float32; activations, and the products' operands, in bf16."""

    def __init__(self, width=256, heads=8, groups=2, dstate=64, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.groups, self.dstate, self.device = heads, groups, dstate, device
        self.inner = heads * HEADDIM
        self.channels = self.inner + 2 * groups * dstate
        rows = self.inner + self.channels + heads          # gate | x B C | step

        def normal(*shape, scale):
            return scale * torch.randn(shape, generator=g, device=device)

        step = torch.exp(torch.empty(heads, device=device).uniform_(-6.9, -2.3, generator=g))   # 0.001 .. 0.1
        self.w = dict(w_in=normal(rows, width, scale=width ** -0.5), w_out=normal(width, self.inner, scale=self.inner ** -0.5),
                      conv=normal(self.channels, 4, scale=0.5), conv_bias=torch.zeros(self.channels, device=device),
                      A=-(1 + 15 * torch.rand(heads, generator=g, device=device)), D=torch.ones(heads, device=device),
                      dt_bias=step + torch.log(-torch.expm1(-step)))

    def split(self, row):
        """Gate, the conv's input and the steps of projected rows (views)."""
        i, c = self.inner, self.channels
        return row[:, :i], row[:, i:i + c], row[:, i + c:]

    def xbc(self, u):
        """x, B and C as parts of the conv's rows (views)."""
        t, i, n = u.shape[0], self.inner, self.groups * self.dstate
        return (u[:, :i].view(t, self.heads, HEADDIM), u[:, i:i + n].view(t, self.groups, self.dstate),
                u[:, i + n:].view(t, self.groups, self.dstate))

    def forward(self, h, cu, max_seqlen, cache=None):
        """Packed tokens (total, width) bf16 -> the same; with ``cache`` from and
        to the requests' caches, without it keeping what backward needs."""
        w = self.w
        row = h @ w["w_in"].bfloat16().t()
        z, xbc, dt = self.split(row)
        ring = {} if cache is None else dict(conv_state=cache["conv"], cache_seqlens=cache["seen"], slots=cache["slots"])
        u = causal_conv1d_varlen_fwd(xbc, w["conv"], cu, bias=w["conv_bias"], activation="silu", **ring)
        x, B, C = self.xbc(u)
        kw = dict(D=w["D"], dt_bias=w["dt_bias"], dt_softplus=True)
        if cache is None:
            entries = ssd_checkpoint_slots(h.shape[0], cu.shape[0] - 1)
            held = (torch.empty(entries, self.heads, HEADDIM, self.dstate, dtype=torch.int8, device=self.device),
                    torch.empty(entries, self.heads, HEADDIM, device=self.device))
            y = ssd_varlen_fwd(x, dt, w["A"], B, C, cu, max_seqlen, checkpoints=held, **kw)
        else:
            held = None
            y = ssd_varlen_fwd(x, dt, w["A"], B, C, cu, max_seqlen, ssm_state=cache["ssm"], cache_seqlens=cache["seen"],
                               slots=cache["slots"], **kw)
            cache["seen"] += cu[1:] - cu[:-1]
        y = y.view(-1, self.inner)
        gated = y * F.silu(z)
        return gated @ w["w_out"].bfloat16().t(), (h, row, u, y, gated, held)

    def backward(self, dout, saved, cu, max_seqlen):
        """Weight gradients of forward (float32)."""
        w = self.w
        h, row, u, y, gated, held = saved
        z, xbc, dt = self.split(row)
        x, B, C = self.xbc(u)
        grads = {"w_out": (dout.t() @ gated).float()}
        dgated = (dout @ w["w_out"].bfloat16()).float()
        zf, yf = z.float(), y.float()
        sig = torch.sigmoid(zf)
        drow, du = torch.empty_like(row), torch.empty_like(u)
        dz, dxbc, ddt = self.split(drow)
        dx, dB, dC = self.xbc(du)
        dz.copy_(dgated * yf * sig * (1 + zf * (1 - sig)))
        dy = (dgated * zf * sig).bfloat16().view_as(x)
        g = ssd_varlen_bwd(x, dt, w["A"], B, C, cu, max_seqlen, dy, held, D=w["D"], dt_bias=w["dt_bias"], dt_softplus=True,
                           dx=dx, dB=dB, dC=dC, ddt=ddt)
        c = causal_conv1d_varlen_bwd(xbc, w["conv"], cu, du, bias=w["conv_bias"], activation="silu", dx=dxbc)
        grads.update(A=g["dA"], D=g["dD"], dt_bias=g["ddt_bias"], conv=c["dweight"], conv_bias=c["dbias"],
                     w_in=(drow.t() @ h).float())
        return grads

    def new_cache(self, entries, requests):
        """Caches of ``entries`` requests; nothing of them is read before it is
        written.  ``requests``: the entries in use, in the batch's order."""
        return dict(conv=torch.empty(entries, self.channels, 4, dtype=torch.bfloat16, device=self.device),
                    ssm=torch.empty(entries, self.heads, HEADDIM, self.dstate, device=self.device),
                    seen=torch.zeros(len(requests), dtype=torch.int32, device=self.device),
                    slots=torch.tensor(requests, dtype=torch.int32, device=self.device))

    def step(self, h, cache):
        """One token of every request: (requests, width) bf16 -> the same."""
        w = self.w
        z, xbc, dt = self.split(h @ w["w_in"].bfloat16().t())
        y = conv1d_ssd_update(xbc, dt, w["A"], w["conv"], cache["conv"], cache["ssm"], cache["seen"],
                              conv_bias=w["conv_bias"], D=w["D"], z=z, dt_bias=w["dt_bias"], dt_softplus=True,
                              slots=cache["slots"])
        cache["seen"] += 1
        return y @ w["w_out"].bfloat16().t()


def packed(lens, device="cuda"):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=device)


def train(mixer, lens=(200, 37, 1, 130), steps=30, rate=3e-3):
    """Losses of a few optimiser steps that teach the mixer a fixed target."""
    g = torch.Generator(device="cuda").manual_seed(7)
    width = mixer.w["w_in"].shape[1]
    h, target = (torch.randn(sum(lens), width, generator=g, device="cuda").bfloat16() for _ in range(2))
    cu, moments, losses = packed(lens), {}, []
    for step in range(1, steps + 1):
        out, saved = mixer.forward(h, cu, max(lens))
        diff = out.float() - 0.5 * target.float()
        losses.append(diff.square().mean().item())
        grads = mixer.backward((2 * diff / diff.numel()).bfloat16(), saved, cu, max(lens))
        for k, v in grads.items():   # Adam
            m, s = moments.setdefault(k, (torch.zeros_like(v), torch.zeros_like(v)))
            m.lerp_(v, 0.1)
            s.lerp_(v.square(), 0.02)
            mixer.w[k] -= rate * (m / (1 - 0.9 ** step)) / ((s / (1 - 0.98 ** step)).sqrt() + 1e-12)
    return losses


def serve(mixer, lens=(70, 5, 129), tokens=6):
    """Outputs of prompts and the tokens after them, and those of the whole
    sequences in one call."""
    g = torch.Generator(device="cuda").manual_seed(8)
    width = mixer.w["w_in"].shape[1]
    whole = [torch.randn(n + tokens, width, generator=g, device="cuda").bfloat16() for n in lens]
    full = [n + tokens for n in lens]
    want, _ = mixer.forward(torch.cat(whole), packed(full), max(full))
    cache = mixer.new_cache(entries=8, requests=[6, 0, 3])
    out, _ = mixer.forward(torch.cat([v[:n] for v, n in zip(whole, lens)]), packed(lens), max(lens), cache)
    got = [list(v) for v in out.split(list(lens))]
    for t in range(tokens):
        y = mixer.step(torch.stack([v[n + t] for v, n in zip(whole, lens)]), cache)
        for s, row in enumerate(y):
            got[s].append(row)
    return torch.cat([torch.stack(v) for v in got]), want


if __name__ == "__main__":
    mixer = Mixer()
    losses = train(mixer)
    print(f"training loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    got, want = serve(mixer)
    off = ((got.float() - want.float()).norm() / want.float().norm()).item()
    print(f"prompts and single tokens against whole sequences: relative difference {off:.2e}")
