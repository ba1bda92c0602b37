"""Experts with block-scaled e4m3 weights, and the routing of tokens to them.

``route_experts`` turns router logits into each token's experts and their weights (softmax or
sigmoid scores, a balance bias on the choice, groups of experts, top-k, renormalisation);
``experts_block_fp8`` runs every token through its experts, gated feed-forward layers whose
three products are those of ``LinearBlockFp8``, and adds the results.  ``RoutedExperts`` is the
layer made of both.

The experts are frozen codes, as ``LinearBlockFp8`` without 16-bit weights: gradients are those
of the input and of the routing weights (and through them of the router), in reverse mode and of the first order alone.
"""
from __future__ import annotations

import contextlib
from typing import Iterable, Optional, Tuple

import torch

from . import abi
from .block import (DTYPES, FixedTypes, _check_input, _dense, _first_order, _no_tangent, _on,
                    _tie, quantize_weight_blocks)


def _route(logits, balance, score, n_groups, top_groups, k, renormalize, scale):
    T = logits.shape[0]
    w = logits.new_empty((T, k), dtype=torch.float32)
    idx = logits.new_empty((T, k), dtype=torch.int32)
    if T > 0:
        with _on(logits.device):
            abi.i8_route_experts(logits, balance, score, n_groups, top_groups, k, renormalize,
                                 scale, w, idx)
    return w, idx


class _RouteFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, balance, score, n_groups, top_groups, k, renormalize, scale):
        w, idx = _route(logits, balance, score, n_groups, top_groups, k, renormalize, scale)
        ctx.save_for_backward(logits, idx)
        ctx.how = (score, renormalize, scale)
        ctx.mark_non_differentiable(idx)
        return w, idx

    @staticmethod
    def backward(ctx, gw, _):
        logits, idx = ctx.saved_tensors
        gl = torch.empty_like(logits)
        if logits.shape[0] > 0:
            with _on(logits.device):
                abi.i8_route_experts_backward(logits, *ctx.how, idx, _dense(gw), gl)
        if torch.is_grad_enabled():
            gl = _first_order(gl, gw, logits)
        return (gl,) + (None,) * 7


def route_experts(logits: torch.Tensor, top_k: int, balance: Optional[torch.Tensor] = None, *,
                  score: str = "softmax", n_groups: int = 1, top_groups: int = 1,
                  renormalize: bool = True,
                  scale: float = 1.0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Each token's `top_k` experts: (weights fp32 [..., k], idx int32 [..., k]).

    logits: fp32, fp16 or bf16 [..., E] on a CUDA device; -inf masks an expert.  balance: fp32
    [E], added to the scores for the choice alone.  A choice that finds no expert left has index
    -1 and weight 0.  The weights are differentiable in the logits.
    """
    if score not in abi.SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    _no_tangent(logits, balance)
    if logits.dim() < 1 or not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor [..., E]")
    E = logits.shape[-1]
    if not 1 <= E <= 512:
        raise ValueError("%d experts: 1 to 512 are supported" % E)
    if not 1 <= top_k <= min(E, 32):
        raise ValueError("top_k %d: 1 to %d are supported" % (top_k, min(E, 32)))
    if not 1 <= n_groups <= 32 or E % n_groups or not 1 <= top_groups <= n_groups:
        raise ValueError("%d of %d groups of %d experts: n_groups divides E and is at most 32, "
                         "top_groups is 1 to n_groups" % (top_groups, n_groups, E))
    if balance is not None:
        if balance.shape != (E,) or balance.dtype != torch.float32:
            raise ValueError("balance must be fp32 [%d]" % E)
        if balance.device != logits.device:
            raise ValueError("balance on %s, logits on %s" % (balance.device, logits.device))
        balance = _dense(balance.detach())
    lead = logits.shape[:-1]
    x = logits if len(lead) == 1 else logits.reshape(-1, E)
    how = (_dense(x), balance, score, n_groups, top_groups, top_k, renormalize, scale)
    if logits.requires_grad and torch.is_grad_enabled():
        w, idx = _RouteFn.apply(*how)
    else:
        w, idx = _route(*how)
    if len(lead) == 1:
        return w, idx
    return w.view(*lead, top_k), idx.view(*lead, top_k)


def _forward(x2, idx, w, CB13, S13, CB2, S2, keep):
    T, K = x2.shape
    E, _, I, _ = CB13.shape
    k = idx.shape[1]
    y = x2.new_empty((T, K))
    gu = w.new_empty((T * k, 2, I)) if keep else None
    if T > 0:
        ws = CB13.new_empty(abi.i8_experts_workspace_size(T, K, I, E, k), dtype=torch.uint8)
        with _on(x2.device):
            abi.i8_experts_forward(x2, idx, w, CB13, S13, CB2, S2, y, gu, ws)
    return y, gu


class _ExpertsFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x2, w, idx, CB13, S13, CB2, S2, tie):
        y, gu = _forward(x2, idx, w, CB13, S13, CB2, S2, True)
        ctx.save_for_backward(w, idx, CB13, S13, CB2, S2, gu)
        ctx.dtype, ctx.tie = x2.dtype, tie[0]
        return y

    @staticmethod
    def backward(ctx, gy):
        w, idx, CB13, S13, CB2, S2, gu = ctx.saved_tensors
        gy = _dense(gy if gy.dtype == ctx.dtype else gy.to(ctx.dtype))
        (T, K), k = gy.shape, idx.shape[1]
        E, _, I, _ = CB13.shape
        gx, gw = torch.empty_like(gy), torch.empty_like(w)
        if T > 0:
            ws = CB13.new_empty(abi.i8_experts_backward_workspace_size(T, K, I, E, k),
                                dtype=torch.uint8)
            with _on(gy.device):
                abi.i8_experts_backward(gy, idx, w, CB13, S13, CB2, S2, gu, gx, gw, ws)
        if torch.is_grad_enabled():
            gx, gw = _first_order(gx, gy, ctx.tie, w), _first_order(gw, gy, ctx.tie)
        return (gx, gw) + (None,) * 6


def experts_block_fp8(x: torch.Tensor, idx: torch.Tensor, weights: torch.Tensor,
                      CB13: torch.Tensor, S13: torch.Tensor, CB2: torch.Tensor,
                      S2: torch.Tensor) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] * W2 (silu(W1 x[t]) * W3 x[t]) with the weights of expert
    idx[t, j]; a negative index is no expert.

    x: fp16 or bf16 [..., K]; idx int32 and weights fp32 [..., k]; CB13 [E, 2, I, K] (W1, W3) and
    CB2 [E, K, I] e4m3 codes with scales S13 [E, 2, ceil(I/128), ceil(K/128)] and S2
    [E, ceil(K/128), ceil(I/128)] (``quantize_weight_blocks``).  Differentiable in x and weights.
    """
    if CB13.dim() != 4:
        raise ValueError("CB13: [E, 2, I, K] codes are required")
    K = CB13.shape[3]
    _check_input(x, K, CB13.device)
    _no_tangent(x, weights, S13, S2)
    for name, t, dtype in (("idx", idx, torch.int32), ("weights", weights, torch.float32)):
        if t.dtype != dtype:
            raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
        if t.dim() < 1 or t.shape[:-1] != x.shape[:-1]:
            raise ValueError("%s of shape %s for an input of shape %s"
                             % (name, tuple(t.shape), tuple(x.shape)))
    if idx.shape != weights.shape:
        raise ValueError("idx of shape %s, weights of shape %s"
                         % (tuple(idx.shape), tuple(weights.shape)))
    k = idx.shape[-1]
    if CB13.shape[0] > 512 or not 1 <= k <= 32:
        raise ValueError("%d experts, %d a token: at most 512 and 1 to 32" % (CB13.shape[0], k))
    x2, i2, w2 = (_dense(t if t.dim() == 2 else t.reshape(-1, t.shape[-1])) for t in (x, idx, weights))
    if torch.is_grad_enabled() and (x2.requires_grad or w2.requires_grad):
        y = _ExpertsFn.apply(x2, w2, i2, CB13, S13, CB2, S2, (_tie(x2),))
    else:
        y, _ = _forward(x2, i2, w2, CB13, S13, CB2, S2, False)
    return y if x.dim() == 2 else y.view(x.shape)


class ExpertsBlockFp8(FixedTypes):
    """E gated feed-forward experts of width `hidden` on `features` features, as block-scaled
    e4m3 codes (buffers ``CB13``, ``S13``, ``CB2``, ``S2``, saved by ``state_dict``; casts of the
    model leave their types alone)."""

    FIXED = ("CB13", "S13", "CB2", "S2")

    def __init__(self, num_experts: int, features: int, hidden: int, device=None):
        super().__init__()
        if not 1 <= num_experts <= 512:
            raise ValueError("%d experts: 1 to 512 are supported" % num_experts)
        if features <= 0 or hidden <= 0 or features % 16 or hidden % 16:
            raise ValueError("features and hidden must be positive multiples of 16 (row pitch of "
                             "the codes for TMA)")
        E, K, I = num_experts, features, hidden
        kb, ib = (K + 127) // 128, (I + 127) // 128
        self.num_experts, self.features, self.hidden = E, K, I
        self.register_buffer("CB13", torch.zeros((E, 2, I, K), dtype=torch.uint8, device=device))
        self.register_buffer("S13", torch.ones((E, 2, ib, kb), dtype=torch.float32, device=device))
        self.register_buffer("CB2", torch.zeros((E, K, I), dtype=torch.uint8, device=device))
        self.register_buffer("S2", torch.ones((E, kb, ib), dtype=torch.float32, device=device))

    @classmethod
    def from_weights(cls, w13: torch.Tensor, w2: torch.Tensor) -> "ExpertsBlockFp8":
        """From fp16 or bf16 weights on a CUDA device: w13 [E, 2, I, K] (gate, then up) and w2
        [E, K, I]."""
        if w13.dim() != 4 or w13.shape[1] != 2 or tuple(w2.shape) != (w13.shape[0], w13.shape[3],
                                                                      w13.shape[2]):
            raise ValueError("w13 [E, 2, I, K] and w2 [E, K, I] are required (got %s, %s)"
                             % (tuple(w13.shape), tuple(w2.shape)))
        m = cls(w13.shape[0], w13.shape[3], w13.shape[2], device=w13.device)
        m.CB13, m.S13 = quantize_weight_blocks(w13)
        m.CB2, m.S2 = quantize_weight_blocks(w2)
        return m

    @classmethod
    def from_linears(cls, gates: Iterable[torch.nn.Linear], ups: Iterable[torch.nn.Linear],
                     downs: Iterable[torch.nn.Linear]) -> "ExpertsBlockFp8":
        """From the experts' nn.Linear layers (without bias, on a CUDA device, one expert after
        another)."""
        gates, ups, downs = list(gates), list(ups), list(downs)
        if not gates or len(gates) != len(ups) or len(gates) != len(downs):
            raise ValueError("%d gate, %d up and %d down layers: the same number of each is "
                             "required" % (len(gates), len(ups), len(downs)))
        if any(m.bias is not None for m in (*gates, *ups, *downs)):
            raise ValueError("experts with a bias are not supported")
        dtype = gates[0].weight.dtype if gates[0].weight.dtype in DTYPES else torch.bfloat16
        w13 = torch.stack([torch.stack([g.weight.detach().to(dtype), u.weight.detach().to(dtype)])
                           for g, u in zip(gates, ups)])
        return cls.from_weights(w13, torch.stack([d.weight.detach().to(dtype) for d in downs]))

    def forward(self, x: torch.Tensor, idx: torch.Tensor, weights: torch.Tensor) -> torch.Tensor:
        return experts_block_fp8(x, idx, weights, self.CB13, self.S13, self.CB2, self.S2)

    def extra_repr(self) -> str:
        return "num_experts=%d, features=%d, hidden=%d" % (self.num_experts, self.features,
                                                           self.hidden)


class RoutedExperts(FixedTypes):
    """A feed-forward layer of experts: router logits x G^T (fp32), route_experts, the experts.

    ``gate``: the router's weight [E, features], a parameter; ``balance``: fp32 [E], a buffer
    that the user's program moves to even out the load, or absent.  Both stay fp32 when the model
    is cast."""

    FIXED = ("gate", "balance")

    def __init__(self, experts: ExpertsBlockFp8, top_k: int, gate: Optional[torch.Tensor] = None,
                 balance: bool = False, score: str = "softmax", n_groups: int = 1,
                 top_groups: int = 1, renormalize: bool = True, scale: float = 1.0):
        super().__init__()
        E, K, dev = experts.num_experts, experts.features, experts.CB13.device
        self.experts = experts
        if gate is not None and tuple(gate.shape) != (E, K):
            raise ValueError("gate of shape %s, expected %s" % (tuple(gate.shape), (E, K)))
        g = torch.zeros((E, K), dtype=torch.float32, device=dev) if gate is None else \
            gate.detach().to(device=dev, dtype=torch.float32).clone()
        self.gate = torch.nn.Parameter(g)
        self.register_buffer("balance", torch.zeros((E,), dtype=torch.float32, device=dev)
                             if balance else None)
        self.top_k = top_k
        self.routing = dict(score=score, n_groups=n_groups, top_groups=top_groups,
                            renormalize=renormalize, scale=scale)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        # near-equal scores decide the choice: no 16-bit product here, under autocast either
        with torch.autocast(x.device.type, enabled=False) \
                if torch.is_autocast_enabled(x.device.type) else contextlib.nullcontext():
            logits = torch.nn.functional.linear(x.float(), self.gate)
        w, idx = route_experts(logits, self.top_k, self.balance, **self.routing)
        return self.experts(x, idx, w)
