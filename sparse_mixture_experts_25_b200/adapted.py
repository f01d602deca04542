"""A sparse MoE layer as it is fine-tuned for many requests and served to them:

    out = residual + dropout(moe(x) + scale_a B_a A_a x),   a = the request's adapter

Training steps run moe_forward, the adapters beside it and the dropout, and
AdaptedLayer.backward gives the gradients of the adapters, of x and of the
layer's own weights.  Serving steps draw nothing and, for at most 32 tokens,
run the layer in its few-token form.  Everything is enqueued on the current
stream of the weights' device, which need not be the current one; tensors of
another device are refused.  The workspaces are the object's, so one object's
calls must not be in flight on two streams at once; they are sized for p.N
tokens, which every call has.
"""
from __future__ import annotations

import functools
from typing import Optional

import torch

from . import (MOE_ACCEPT_TOKEN, MOE_OK, MOE_REJECT_REROUTE, MoEError, adapter_params, dropout_params,
               moe_adapter_backward, moe_adapter_backward_workspace_size, moe_adapter_check, moe_adapter_forward,
               moe_adapter_workspace_size, moe_backward, moe_backward_check, moe_backward_workspace_size,
               moe_dropout_backward, moe_dropout_forward, moe_few_workspace_size, moe_forward, moe_forward_few,
               moe_get_stats, moe_workspace_size, workspace_views)

FEW_TOKENS = 32
WEIGHTS = ("W_r", "b_r", "W_g", "W_u", "W_d", "Ws_g", "Ws_u", "Ws_d")


def _on_its_device(method):
    """Runs a method of an AdaptedLayer with the layer's device current: what it
    calls is launched on the current device."""

    @functools.wraps(method)
    def call(self, *args, **kw):
        with torch.cuda.device(self.device):
            return method(self, *args, **kw)

    return call


class AdaptedLayer:
    """The layer of `p` (moe.params) with `n_adapters` adapters of rank `r` and
    dropout of `rate` under `seed`.

    weights: dict of the layer's tensors (WEIGHTS; b_r and the shared expert's
    may be missing).  A [n_adapters, r, d], B [n_adapters, d, r] of the layer's
    dtype, scale [n_adapters] fp32."""

    def __init__(self, p, weights, A, B, scale, rate: float = 0.0, seed: int = 0):
        self.p, self.A, self.B, self.scale = p, A, B, scale
        self.w = {n: weights.get(n) for n in WEIGHTS}
        n_adapters, r = A.shape[:2]
        self.ap = adapter_params(p.N, p.d, p.d, n_adapters, r, dtype=p.dtype)
        self.rate, self.seed = rate, seed
        self.device = dev = A.device
        self._same_device(B=B, scale=scale, **self.w)
        # what the few-token form covers
        self.few = (p.N <= FEW_TOKENS and p.E_r <= 256 and p.reject_policy != MOE_REJECT_REROUTE
                    and p.accept_order == MOE_ACCEPT_TOKEN and p.E_r * p.d_f + p.d_f_shared < 1 << 24)
        size = max(moe_workspace_size(p), moe_few_workspace_size(p) if self.few else 0)
        self.ws = torch.empty(size, dtype=torch.uint8, device=dev)
        self.aws = torch.empty(moe_adapter_workspace_size(self.ap), dtype=torch.uint8, device=dev)
        self.Y = torch.empty(p.N, p.d, dtype=torch.float32, device=dev)
        self.bws: Optional[torch.Tensor] = None
        self.abws: Optional[torch.Tensor] = None
        self.saved = None
        self.called = False  # until then the workspaces hold nothing

    def _same_device(self, **tensors):
        for n, t in tensors.items():
            if t is not None and t.device != self.device:
                raise ValueError(f"{n}: expected a tensor on {self.device}, got {t.device}")

    def _drop(self, rate, offset, row0):
        return dropout_params(self.p.N, self.p.d, rate, seed=self.seed, offset=offset, row0=row0, dtype=self.p.dtype)

    @_on_its_device
    def forward(self, x, ids, residual, lat=None, training: bool = False, offset: int = 0, row0: int = 0):
        """out [N, d] of the layer's dtype.  ids [N] int32 (-1: no adapter).
        training: draws the dropout of call `offset` (row0: the first token's
        row in a sharded batch) and keeps what backward needs."""
        self._same_device(x=x, ids=ids, residual=residual, lat=lat)
        w = self.w
        call = moe_forward if training or not self.few else moe_forward_few
        call(self.p, x, w["W_r"], w["b_r"], lat, w["W_g"], w["W_u"], w["W_d"], w["Ws_g"], w["Ws_u"], w["Ws_d"],
             self.Y, self.ws)
        moe_adapter_forward(self.ap, x, None, self.A, self.B, self.scale, ids, self.Y, self.Y, self.aws)
        out = torch.empty(self.p.N, self.p.d, dtype=x.dtype, device=x.device)
        dp = self._drop(self.rate if training else 0.0, offset, row0)
        moe_dropout_forward(dp, self.Y, residual, out)
        self.saved = (x, ids, dp) if training else None
        self.called = True
        return out

    @_on_its_device
    def backward(self, dout, aux_coef: float = 0.0):
        """Gradients for dout [N, d] of the layer's dtype, of the last training
        forward: a dict of fp32 tensors (dA, dB, dx and moe_backward's weight
        gradients; the residual's gradient is dout).  Reads the forward's row
        counts back to the host, so it waits for the forward.  No other step of
        this object may run between the two, a replayed one neither: the
        workspaces are the object's."""
        if self.saved is None:
            raise ValueError("backward follows a training forward")
        self._same_device(dout=dout)
        x, ids, dp = self.saved
        p, w, dev = self.p, self.w, x.device

        def empty(t):
            return torch.empty(t.shape, dtype=torch.float32, device=dev)

        dY = empty(self.Y)
        moe_dropout_backward(dp, dout, dY)
        offsets = workspace_views(p, self.ws)["offsets"].cpu().numpy()
        size = moe_backward_workspace_size(p, offsets)
        if self.bws is None or self.bws.numel() < size:
            self.bws = torch.empty(size, dtype=torch.uint8, device=dev)
        if self.abws is None:
            self.abws = torch.empty(moe_adapter_backward_workspace_size(self.ap), dtype=torch.uint8, device=dev)
        grads = {"dx": empty(self.Y), **{"d" + n: empty(t) for n, t in w.items() if t is not None}}
        moe_backward(p, offsets, x, w["W_r"], w["b_r"], w["W_g"], w["W_u"], w["W_d"], w["Ws_g"], w["Ws_u"], w["Ws_d"],
                     dY, self.ws, grads, self.bws, aux_coef=aux_coef)
        grads.update(dA=empty(self.A), dB=empty(self.B))
        moe_adapter_backward(self.ap, x, None, self.A, self.B, self.scale, ids, dY, grads["dx"], grads["dx"],
                             grads["dA"], grads["dB"], self.abws)
        return grads

    @_on_its_device
    def check(self):
        """Waits for the current stream and raises what the last forward (and
        backward) reported: tokens with non-finite scores, ids out of range, a
        bounded wait that gave up.  Returns the routing statistics."""
        if not self.called:
            raise ValueError("check follows a forward")
        status, stats = moe_get_stats(self.p, self.ws)
        found = [(status, "layer"), (moe_adapter_check(self.ap, self.aws), "adapters")]
        if self.bws is not None:
            found += [(moe_backward_check(self.p, self.bws), "layer gradients"),
                      (moe_adapter_check(self.ap, self.abws), "adapter gradients")]
        for s, where in found:
            if s != MOE_OK:
                raise MoEError(s, where)
        return stats
