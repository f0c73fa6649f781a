"""A gated recurrent block trained and served with the packed-token operators.

    python examples/gated_block.py

The residual stream (float32) takes the branch before it and is normed in one
call (rms_norm_fwd); the input projection gives a gate and the recurrence's
input, which goes through the short convolution (causal_conv1d_varlen_fwd), the
gates' projection and the gated linear recurrence (gated_scan_varlen_fwd); the
gated norm and the output projection make the next branch.  Training runs back
through rms_norm_bwd, gated_scan_varlen_bwd and causal_conv1d_varlen_bwd; serving
fills the requests' caches with prompts of several lengths in one call and adds a
token to each of them with gated_scan_update.  Random weights and data.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from state_space_model_scan_amd import (causal_conv1d_varlen_bwd, causal_conv1d_varlen_fwd, gated_checkpoint_slots,  # noqa: E402
                                        gated_scan_update, gated_scan_varlen_bwd, gated_scan_varlen_fwd, rms_norm_bwd,
                                        rms_norm_fwd)


class Block:
    """Weights in float32; the branch's activations, and the products' operands,
    in bf16."""

    def __init__(self, width=256, inner=384, groups=3, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.inner, self.group, self.device = inner, inner // groups, device

        def normal(*shape, scale):
            return scale * torch.randn(shape, generator=g, device=device)

        decay = torch.empty(inner, device=device).uniform_(0.9, 0.999, generator=g)
        self.w = dict(norm=torch.ones(width, device=device), w_in=normal(2 * inner, width, scale=width ** -0.5),
                      conv=normal(inner, 4, scale=0.5), conv_bias=torch.zeros(inner, device=device),
                      w_gates=normal(2 * inner, inner, scale=inner ** -0.5), r_bias=torch.zeros(inner, device=device),
                      i_bias=torch.zeros(inner, device=device), A=8 * torch.log(decay),
                      gated_norm=torch.ones(inner, device=device), w_out=normal(width, inner, scale=inner ** -0.5))

    def forward(self, branch, stream, cu, cache=None):
        """(branch (tokens, width) bf16, residual stream (tokens, width) float32) ->
        the same and what backward needs; with ``cache`` from and to the requests'
        caches, ``cu`` None for a single token of each."""
        w, i = self.w, self.inner
        normed, stream = rms_norm_fwd(branch, w["norm"], residual=stream)
        row = normed @ w["w_in"].bfloat16().t()
        z, x = row[:, :i], row[:, i:]
        one = cu is None
        edges = cache["each"] if one else cu
        ring = {} if cache is None else dict(conv_state=cache["conv"], cache_seqlens=cache["seen"], slots=cache["slots"])
        u = causal_conv1d_varlen_fwd(x, w["conv"], edges, bias=w["conv_bias"], **ring)
        gates = u @ w["w_gates"].bfloat16().t()
        r, g = gates[:, :i], gates[:, i:]
        kw = dict(r_bias=w["r_bias"], i_bias=w["i_bias"])
        held = None
        if cache is None:
            held = torch.empty(gated_checkpoint_slots(u.shape[0]), i, device=self.device)
            h = gated_scan_varlen_fwd(u, r, g, w["A"], cu, checkpoints=held, **kw)
        elif one:
            h = gated_scan_update(u, r, g, w["A"], cache["state"], cache["seen"], slots=cache["slots"], **kw)
        else:
            h = gated_scan_varlen_fwd(u, r, g, w["A"], cu, state=cache["state"], cache_seqlens=cache["seen"],
                                      slots=cache["slots"], **kw)
        if cache is not None:
            cache["seen"] += 1 if one else cu[1:] - cu[:-1]
        out = rms_norm_fwd(h, w["gated_norm"], z=z, group_size=self.group)
        return out @ w["w_out"].bfloat16().t(), stream, (normed, stream, row, u, gates, held, h, out)

    def backward(self, dbranch, dstream, saved, cu):
        """Gradients of the weights (float32), of the branch (bf16) and of the
        stream (float32) that went in."""
        w, i = self.w, self.inner
        normed, stream, row, u, gates, held, h, out = saved
        z, x = row[:, :i], row[:, i:]
        r, g = gates[:, :i], gates[:, i:]
        grads = {"w_out": (dbranch.t() @ out).float()}
        drow, dgates = torch.empty_like(row), torch.empty_like(gates)
        n = rms_norm_bwd(h, w["gated_norm"], dbranch @ w["w_out"].bfloat16(), z=z, group_size=self.group, dz=drow[:, :i])
        s = gated_scan_varlen_bwd(u, r, g, w["A"], cu, n["dx"], held, r_bias=w["r_bias"], i_bias=w["i_bias"],
                                  dr=dgates[:, :i], di=dgates[:, i:])
        du = s["dx"] + dgates @ w["w_gates"].bfloat16()
        c = causal_conv1d_varlen_bwd(x, w["conv"], cu, du, bias=w["conv_bias"], dx=drow[:, i:])
        first = rms_norm_bwd(stream, w["norm"], drow @ w["w_in"].bfloat16(), ds=dstream)
        grads.update(gated_norm=n["dweight"], A=s["dA"], r_bias=s["dr_bias"], i_bias=s["di_bias"],
                     w_gates=(dgates.t() @ u).float(), conv=c["dweight"], conv_bias=c["dbias"],
                     w_in=(drow.t() @ normed).float(), norm=first["dweight"])
        return grads, first["dx"], first["dresidual"]

    def new_cache(self, entries, requests):
        """Caches of ``entries`` requests; nothing of them is read before it is
        written.  ``requests``: the entries in use, in the batch's order."""
        n = len(requests)
        return dict(conv=torch.empty(entries, self.inner, 4, dtype=torch.bfloat16, device=self.device),
                    state=torch.empty(entries, self.inner, device=self.device),
                    seen=torch.zeros(n, dtype=torch.int32, device=self.device),
                    slots=torch.tensor(requests, dtype=torch.int32, device=self.device),
                    each=torch.arange(n + 1, dtype=torch.int32, device=self.device))


def packed(lens, device="cuda"):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=device)


def data(lens, width, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(sum(lens), width, generator=g, device="cuda") for _ in range(3)]


def train(block, lens=(200, 37, 1, 130), steps=30, rate=3e-3):
    """Losses of a few optimiser steps that teach the block a fixed target."""
    width = block.w["norm"].shape[0]
    branch, stream, target = data(lens, width, 7)
    branch, cu, moments, losses = branch.bfloat16(), packed(lens), {}, []
    for step in range(1, steps + 1):
        out, held, saved = block.forward(branch, stream, cu)
        diff = out.float() + held - stream - 0.5 * target
        losses.append(diff.square().mean().item())
        grad = 2 * diff / diff.numel()
        grads, _, _ = block.backward(grad.bfloat16(), grad, saved, cu)
        for k, v in grads.items():   # Adam
            m, s = moments.setdefault(k, (torch.zeros_like(v), torch.zeros_like(v)))
            m.lerp_(v, 0.1)
            s.lerp_(v.square(), 0.02)
            block.w[k] -= rate * (m / (1 - 0.9 ** step)) / ((s / (1 - 0.98 ** step)).sqrt() + 1e-12)
        block.w["A"].clamp_(max=-1e-6)
    return losses


def serve(block, lens=(70, 5, 129), tokens=6):
    """Outputs of prompts and the tokens after them, and those of the whole
    sequences in one call."""
    width = block.w["norm"].shape[0]
    full = [n + tokens for n in lens]
    branch, stream, _ = data(full, width, 8)
    branch, cu = branch.bfloat16(), packed(full)
    want, _, _ = block.forward(branch, stream, cu)
    at = cu.tolist()
    cache = block.new_cache(entries=8, requests=[6, 0, 3])
    rows = torch.cat([torch.arange(a, a + n) for a, n in zip(at, lens)]).cuda()
    out, _, _ = block.forward(branch[rows], stream[rows], packed(lens), cache)
    got = [list(v) for v in out.split(list(lens))]
    for t in range(tokens):
        rows = torch.tensor([a + n + t for a, n in zip(at, lens)]).cuda()
        out, _, _ = block.forward(branch[rows], stream[rows], None, cache)
        for s, row in enumerate(out):
            got[s].append(row)
    return torch.cat([torch.stack(v) for v in got]), want


if __name__ == "__main__":
    block = Block()
    losses = train(block)
    print(f"training loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    got, want = serve(block)
    off = ((got.float() - want.float()).norm() / want.float().norm()).item()
    print(f"prompts and single tokens against whole sequences: relative difference {off:.2e}")
