"""Python binding of a gated recurrent block's operators: its recurrence over
packed tokens, its single-token step, and its norm.

The checks and the marshalling are in C++ (csrc/packed_binding.cpp); each
function there returns a status first.  A ``stream`` other than the current one
takes the whole call, and the caller orders it after what made the inputs.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from ._lib import check


def handle(stream) -> Optional[int]:
    return None if stream is None else stream.cuda_stream


def gated_checkpoint_slots(total: int) -> int:
    """Kept states of ``total`` packed tokens."""
    return -(-total // _lib.GATED_CHUNK)


def gated_scan_varlen_fwd(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, A: torch.Tensor, cu_seqlens: torch.Tensor,
                          r_bias: Optional[torch.Tensor] = None, i_bias: Optional[torch.Tensor] = None,
                          state: Optional[torch.Tensor] = None, cache_seqlens: Optional[torch.Tensor] = None,
                          slots: Optional[torch.Tensor] = None, checkpoints: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Gated linear recurrence over packed tokens; returns ``out`` (total,
    channels): a state h <- a h + sqrt(1 - a^2) sigmoid(i + i_bias) x for every
    sequence and channel, with a = exp(A sigmoid(r + r_bias)).

    x, r, i: (total, channels), any token stride; A (<= 0), r_bias, i_bias:
    (channels,) float32; cu_seqlens: (nseq + 1,) int32.  ``state`` (entries,
    channels) float32 is the requests' cache, read where ``cache_seqlens[s]`` > 0
    and written, at entry ``slots[s]`` (s without ``slots``; an entry outside the
    cache is skipped).  ``checkpoints`` (gated_checkpoint_slots(total), channels)
    float32 receives what gated_scan_varlen_bwd starts from.  Tokens before
    cu_seqlens[0] or from cu_seqlens[nseq] on are padding: their rows of ``out``
    are left as they were."""
    status, out = _lib.packed().gated_fwd(x, r, i, A, cu_seqlens, r_bias, i_bias, state, cache_seqlens, slots, checkpoints, out,
                                          workspace, handle(stream))
    if status:
        check(status)
    return out


def gated_scan_varlen_bwd(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, A: torch.Tensor, cu_seqlens: torch.Tensor,
                          dout: torch.Tensor, checkpoints: torch.Tensor, r_bias: Optional[torch.Tensor] = None,
                          i_bias: Optional[torch.Tensor] = None, initial_states: Optional[torch.Tensor] = None,
                          dfinal_states: Optional[torch.Tensor] = None, want_dinitial_states: bool = False,
                          dx: Optional[torch.Tensor] = None, dr: Optional[torch.Tensor] = None,
                          di: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          stream=None) -> dict:
    """Gradients of gated_scan_varlen_fwd in a dict: dx, dr and di in x's dtype
    (into the tensors given, which may be parts of one row, or new ones; 0 for
    padding), dA, dr_bias and di_bias in float32.

    ``checkpoints``: what the forward wrote.  ``initial_states`` (nseq, channels)
    float32: the states that the sequences started from (None: zero);
    ``dfinal_states``, of the same shape, the gradient of their last ones.  With
    ``want_dinitial_states`` that of the first ones is returned."""
    if checkpoints is None:
        raise ValueError("the backward needs the checkpoints that the forward wrote")
    status, *grads = _lib.packed().gated_bwd(x, r, i, A, cu_seqlens, dout, checkpoints, r_bias, i_bias, initial_states,
                                             dfinal_states, want_dinitial_states, dx, dr, di, workspace, handle(stream))
    if status:
        check(status)
    names = ("dx", "dr", "di", "dA", "dr_bias", "di_bias", "dinitial_states")
    return {k: v for k, v in zip(names, grads) if v is not None}


def gated_scan_update(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, A: torch.Tensor, state: torch.Tensor,
                      cache_seqlens: Optional[torch.Tensor], r_bias: Optional[torch.Tensor] = None,
                      i_bias: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of every request through gated_scan_varlen_fwd's recurrence;
    returns ``out`` (batch, channels).

    x, r, i: (batch, channels), any row stride; ``state`` (entries, channels)
    float32 is the cache that gated_scan_varlen_fwd fills, updated in place;
    request b uses entry ``slots[b]`` and has seen ``cache_seqlens[b]`` tokens
    (None: every request is new).  A row whose entry is outside the cache is
    padding."""
    status, out = _lib.packed().gated_step(x, r, i, A, state, cache_seqlens, r_bias, i_bias, slots, out, handle(stream))
    if status:
        check(status)
    return out


def rms_norm_fwd(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                 z: Optional[torch.Tensor] = None, group_size: Optional[int] = None, eps: float = 1e-5,
                 out: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None, stream=None):
    """Root-mean-square norm of x, of x + ``residual`` or of x silu(``z``), over
    groups of ``group_size`` neighbouring columns (None: the row), times
    ``weight``; returns ``out``, or (``out``, ``residual_out``) with a residual.

    x, z: (rows, cols), any row stride; weight: (cols,) float32; residual: (rows,
    cols) in x's dtype or float32.  ``residual_out`` holds x + residual in its
    dtype (it may be ``residual`` itself), and is what is normalised."""
    status, out, _, residual_out = _lib.packed().norm_fwd(x, weight, residual, z, group_size, eps, False, out, None, residual_out,
                                                          handle(stream))
    if status:
        check(status)
    return out if residual_out is None else (out, residual_out)


def rms_norm_quant_fwd(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                       z: Optional[torch.Tensor] = None, group_size: Optional[int] = None, eps: float = 1e-5,
                       codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                       residual_out: Optional[torch.Tensor] = None, stream=None):
    """rms_norm_fwd to 8 bits; returns (``codes``, ``scales``), or (``codes``,
    ``scales``, ``residual_out``) with a residual.

    codes: (rows, cols) float8_e4m3fn; scales: (rows, ceil(cols / 128)) float32,
    one power of two for 128 columns of a row: the value is code * scale.  More
    than one group a row takes a ``group_size`` that is a multiple of 128."""
    status, codes, scales, residual_out = _lib.packed().norm_fwd(x, weight, residual, z, group_size, eps, True, codes, scales,
                                                                 residual_out, handle(stream))
    if status:
        check(status)
    return (codes, scales) if residual_out is None else (codes, scales, residual_out)


def rms_norm_bwd(x: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor, z: Optional[torch.Tensor] = None,
                 ds: Optional[torch.Tensor] = None, group_size: Optional[int] = None, eps: float = 1e-5,
                 dx: Optional[torch.Tensor] = None, dresidual: Optional[torch.Tensor] = None,
                 dz: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of rms_norm_fwd in a dict.

    ``x``: the forward's x, or with a residual its ``residual_out``; ``dy``: the
    output's gradient; ``ds`` (x's dtype): with a residual, the gradient that
    reaches ``residual_out`` from elsewhere.  dx, the gradient of x and of the
    residual, comes in dy's dtype, and where x's is another in that too, as
    dresidual; dz in dy's dtype, dweight in float32."""
    status, dx, dresidual, dz, dweight = _lib.packed().norm_bwd(x, weight, dy, z, ds, group_size, eps, dx, dresidual, dz,
                                                                workspace, handle(stream))
    if status:
        check(status)
    return {k: v for k, v in (("dx", dx), ("dresidual", dresidual), ("dz", dz), ("dweight", dweight)) if v is not None}
