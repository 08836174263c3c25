"""The time mix's operators as differentiable torch functions.

    y, state = autograd.wkv(k, v, w, u, r, state_in)
    xk, xv, xr, x_last = autograd.token_shift(x, mix_k, mix_v, mix_r, x_prev)

The forward and the gradients run in the library's kernels
(``wkv4.forward`` / ``forward_gated`` / ``token_shift`` and ``wkv4.backward`` /
``token_shift_backward``); a call keeps its inputs (and the state it returned)
for the backward pass and recomputes the rest there.  What it kept must not be
changed before then: ``wkv4.decode_step`` on a state that still has a backward
pass to come takes a clone.  Gradients are those of first order only.

The state's max plane fixes the unit its sums are held in; a gradient that
arrives for it is not read (see ``wkv4_backward`` in include/wkv4.h).

A forward and backward pass can be captured into a CUDA graph as torch's own
operators can: warmed up and captured on a side stream, and only while no eager
graph of the same leaves lives (drop its loss and outputs first).  torch ties
a leaf's gradient to the stream of the graph that used it first, and a capture
that would wait for that stream is refused by CUDA.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import wkv4


def _grad(g: Optional[torch.Tensor], like: torch.Tensor) -> torch.Tensor:
    return torch.zeros_like(like) if g is None else g.contiguous()


class _Wkv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, k, v, w, u, r, state_in):
        if r is None:
            y, state = wkv4.forward(k, v, w, u, state_in)
        else:
            y, state = wkv4.forward_gated(k, v, r, w, u, state_in)
        ctx.save_for_backward(k, v, w, u, r, state_in, state)
        ctx.set_materialize_grads(False)
        return y, state

    @staticmethod
    @once_differentiable
    def backward(ctx, gy, gstate):
        k, v, w, u, r, state_in, state = ctx.saved_tensors
        if gy is None and gstate is None:
            return (None,) * 6
        g = wkv4.backward(k, v, w, u, _grad(gy, k), state_in, r=r,
                          state_out=None if gstate is None else state,
                          gstate_out=None if gstate is None else gstate.contiguous())
        return g.gk, g.gv, g.gw, g.gu, g.gr, g.gstate_in


def wkv(k: torch.Tensor, v: torch.Tensor, w: torch.Tensor, u: torch.Tensor,
        r: Optional[torch.Tensor] = None,
        state_in: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``wkv4.forward`` (with r: ``wkv4.forward_gated``), differentiable by every
    tensor given.  Returns (y, state after the last step)."""
    return _Wkv.apply(k, v, w, u, r, state_in)


class _TokenShift(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, mix_k, mix_v, mix_r, x_prev):
        x_last = torch.empty((x.shape[0], x.shape[2]), dtype=x.dtype, device=x.device)
        xk, xv, xr = wkv4.token_shift(x, mix_k, mix_v, mix_r, x_prev, x_last=x_last)
        ctx.save_for_backward(x, mix_k, mix_v, mix_r, x_prev)
        ctx.set_materialize_grads(False)
        return xk, xv, xr, x_last

    @staticmethod
    @once_differentiable
    def backward(ctx, gxk, gxv, gxr, gx_last):
        x, mix_k, mix_v, mix_r, x_prev = ctx.saved_tensors
        if gxk is None and gxv is None and gxr is None and gx_last is None:
            return (None,) * 5
        g = wkv4.token_shift_backward(x, mix_k, mix_v, _grad(gxk, x), _grad(gxv, x), mix_r,
                                      None if mix_r is None else _grad(gxr, x), x_prev,
                                      gx_last=None if gx_last is None else gx_last.contiguous())
        return g.gx, g.gmix_k, g.gmix_v, g.gmix_r, g.gx_prev


def token_shift(x: torch.Tensor, mix_k: torch.Tensor, mix_v: torch.Tensor,
                mix_r: Optional[torch.Tensor] = None, x_prev: Optional[torch.Tensor] = None):
    """``wkv4.token_shift``, differentiable by every tensor given.  Returns
    (xk, xv, xr or None, x_last), x_last [B, C] the next call's x_prev."""
    return _TokenShift.apply(x, mix_k, mix_v, mix_r, x_prev)
