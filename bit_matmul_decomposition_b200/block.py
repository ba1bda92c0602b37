"""Linear layers with block-scaled e4m3 codes: one fp32 scale for each 128 x 128 tile of the
weight and for each 128 features of a token.

Where ``Linear8bitLt`` keeps one scale per row and takes the outlier columns out into an fp16
product, a block's scale confines an outlier to its block, so every feature goes through the
8-bit product.  The weight format (e4m3 codes and a scale tensor of one entry per 128 x 128
tile, value = code * scale) is that of checkpoints stored in it: ``LinearBlockFp8.from_codes``
takes them as they are.

Activations and bias are fp16 or bf16; the output has their type.  Any number of tokens runs in
the library's kernels (i8_block_linear_forward): few tokens stream the weight once, more take the
tensor-core tiles.

Gradients pass straight through the quantisation, in the same 8-bit products
(i8_block_linear_backward): dx = q(dy) W' with dy in blocks of 128 per token, and for a layer
that trains its 16-bit weight dW = t(dy)^T t(x) in 128 x 128 tiles, db = sum(dy).  There is no
forward-mode derivative (a dual tensor is refused) and no second one (create_graph gives the same
gradients, and differentiating them again raises).
"""
from __future__ import annotations

import contextlib
from typing import Iterable, Optional, Tuple

import torch
from torch.autograd import forward_ad

from . import abi

DTYPES = (torch.float16, torch.bfloat16)


def _on(device: torch.device):
    """Makes `device` current, for the library launches there; nothing where it is already."""
    if device.index == torch.cuda.current_device():
        return _HERE
    return torch.cuda.device(device)


_HERE = contextlib.nullcontext()


def _dense(t: torch.Tensor) -> torch.Tensor:
    """Contiguous and on a 16-byte boundary, as the library takes its pointers."""
    if not t.is_contiguous():
        t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _no_tangent(*tensors):
    """Refuses forward-mode dual tensors: a library call fills a fresh buffer, which would have
    no tangent, and so a derivative of zero."""
    if forward_ad._current_level < 0:       # no dual_level() is open: no dual tensor (1 us saved)
        return
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError("no forward-mode derivative: the library's layers have "
                                      "gradients (reverse mode) alone")


class _FirstOrder(torch.autograd.Function):
    @staticmethod
    def forward(ctx, grad, *depends):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, _):
        raise NotImplementedError("no second derivative: the library's layers have first-order "
                                  "gradients alone")


def _first_order(grad, *depends):
    """A gradient on its way out of a backward that the library computed, under create_graph (the
    only time that gradients are enabled in a backward).  It is tied to the tensors of the graph
    that it depends on, so that differentiating it again raises; without the tie its terms would
    be missing from the sum and no error seen.  (torch.autograd.function.once_differentiable ties
    it to the gradients that came in alone: a constant one, as sum() gives, leaves nothing to
    raise.)"""
    if grad is None:
        return None
    depends = [t for t in depends if t is not None and t.requires_grad]
    return _FirstOrder.apply(grad, *depends) if depends else grad


def _tie(t):
    """For a tensor that a backward does not read: what `_first_order` needs of it.  A leaf itself,
    or an empty tensor with the history of `t` but none of its memory."""
    if not t.requires_grad or t.is_leaf:
        return t if t.requires_grad else None
    return torch.slice_copy(t, 0, 0, 0)


def _check_input(x: torch.Tensor, K: int, device: torch.device, name: str = "input"):
    if x.dtype not in DTYPES:
        raise TypeError("%s must be fp16 or bf16 (got %s)" % (name, x.dtype))
    if x.dim() < 1 or x.shape[-1] != K:
        raise ValueError("last %s dimension %s, expected %d"
                         % (name, x.shape[-1] if x.dim() else "missing", K))
    if x.device != device:
        raise ValueError("%s on %s, layer on %s" % (name, x.device, device))


def quantize_weight_blocks(weight: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """e4m3 codes (uint8, the shape of `weight` [..., N, K]) and scales [..., ceil(N/128),
    ceil(K/128)] of an fp16 or bf16 weight on a CUDA device."""
    if not weight.is_cuda:
        raise ValueError("the weight must be on a CUDA device (it is quantised there)")
    if weight.dtype not in DTYPES:
        raise TypeError("the weight must be fp16 or bf16 (got %s)" % weight.dtype)
    w = _dense(weight.detach())
    N, K = w.shape[-2:]
    codes = w.new_empty(w.shape, dtype=torch.uint8)
    scales = w.new_empty((*w.shape[:-2], (N + 127) // 128, (K + 127) // 128), dtype=torch.float32)
    with _on(w.device):
        abi.i8_block_quantize_weight(w, codes, scales)
    return codes, scales


def _forward(x2, codes, scales, bias):
    T, K = x2.shape
    N = codes.shape[0]
    y = x2.new_empty((T, N))
    if T > 0:
        # the workspace is the caching allocator's: ordered by the stream, and a graph that is
        # being captured gets one of its own
        ws = codes.new_empty(abi.i8_block_linear_workspace_size(T, N, K), dtype=torch.uint8)
        with _on(x2.device):
            abi.i8_block_linear_forward(x2, codes, scales, bias, y, ws)
    return y


def _backward(gy, x2, codes, scales, K, want_x, want_w, want_b, dtype):
    gy = _dense(gy if gy.dtype == dtype else gy.to(dtype))
    T, N = gy.shape
    new = gy.new_zeros if T == 0 else gy.new_empty
    gx = new((T, K)) if want_x else None
    gw = new((N, K)) if want_w else None
    gb = new((N,)) if want_b else None
    if T > 0 and (want_x or want_w or want_b):
        ws = gy.new_empty(abi.i8_block_linear_backward_workspace_size(T, N, K), dtype=torch.uint8)
        with _on(gy.device):
            abi.i8_block_linear_backward(gy, x2, codes, scales, gx, gw, gb, ws)
    return gx, gw, gb


class _BlockLinearFn(torch.autograd.Function):
    """Frozen codes: gradients of the input and of the bias."""

    @staticmethod
    def forward(ctx, x2, codes, scales, bias):
        ctx.save_for_backward(codes, scales)
        ctx.dtype = x2.dtype
        return _forward(x2, codes, scales, bias)

    @staticmethod
    def backward(ctx, gy):
        codes, scales = ctx.saved_tensors
        gx, _, gb = _backward(gy, None, codes, scales, codes.shape[1], ctx.needs_input_grad[0],
                              False, ctx.needs_input_grad[3], ctx.dtype)
        if torch.is_grad_enabled():
            gx, gb = _first_order(gx, gy), _first_order(gb, gy)
        return gx, None, None, gb


class _BlockLinearTrainFn(torch.autograd.Function):
    """A 16-bit weight, quantised by every forward: gradients of input, weight and bias."""

    @staticmethod
    def forward(ctx, x2, weight, bias, tie):
        codes, scales = quantize_weight_blocks(weight)
        ctx.save_for_backward(x2, codes, scales)
        ctx.tie = tie[0]
        return _forward(x2, codes, scales, bias)

    @staticmethod
    def backward(ctx, gy):
        x2, codes, scales = ctx.saved_tensors
        gx, gw, gb = _backward(gy, x2, codes, scales, codes.shape[1], *ctx.needs_input_grad[:3],
                               x2.dtype)
        if torch.is_grad_enabled():
            gx, gw, gb = _first_order(gx, gy, ctx.tie), _first_order(gw, gy, x2), _first_order(gb, gy)
        return gx, gw, gb, None


def linear_block_fp8(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                     bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = x W^T + bias with W given as e4m3 codes [N, K] (uint8 or float8_e4m3fn) and scales
    [ceil(N/128), ceil(K/128)].  x: fp16 or bf16 [..., K], bias: x's type [N].  Differentiable in x
    and bias; codes and scales are constants."""
    if codes.dim() != 2:
        raise ValueError("codes: a 2-D tensor is required")
    _check_input(x, codes.shape[1], codes.device)
    _no_tangent(x, scales, bias)
    x2 = _dense(x if x.dim() == 2 else x.reshape(-1, codes.shape[1]))
    if torch.is_grad_enabled() and (x2.requires_grad or (bias is not None and bias.requires_grad)):
        y = _BlockLinearFn.apply(x2, codes, scales, bias)
    else:
        y = _forward(x2, codes, scales, bias)
    return y if x.dim() == 2 else y.view(*x.shape[:-1], codes.shape[0])


def linear_block_fp8_train(x: torch.Tensor, weight: torch.Tensor,
                           bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = x W^T + bias, the 16-bit weight [N, K] quantised in 128 x 128 tiles by this call;
    differentiable in x, weight and bias (all of one type, fp16 or bf16)."""
    if weight.dim() != 2:
        raise ValueError("weight: a 2-D tensor is required")
    _check_input(x, weight.shape[1], weight.device)
    if weight.dtype != x.dtype:
        raise TypeError("weight is %s, input %s: one type is required" % (weight.dtype, x.dtype))
    _no_tangent(x, weight, bias)
    x2 = _dense(x if x.dim() == 2 else x.reshape(-1, weight.shape[1]))
    y = _BlockLinearTrainFn.apply(x2, weight, bias, (_tie(weight),))
    return y if x.dim() == 2 else y.view(*x.shape[:-1], weight.shape[0])


class FixedTypes(torch.nn.Module):
    """A module some of whose tensors have the one type that the library takes: casts of the
    model (``.half()``, ``.to(torch.bfloat16)``, ``.double()``) move them, but leave type, values and
    layout alone.  Cast, the scales would lose bits for good, and fp16 holds few of them at all."""

    FIXED: Tuple[str, ...] = ()                # names of such buffers and parameters

    def _apply(self, fn, recurse=True):
        if recurse:
            for child in self.children():
                child._apply(fn)
        fixed = [t for t in (getattr(self, name, None) for name in self.FIXED) if t is not None]
        fixed += [t.grad for t in fixed if t.grad is not None]

        def keep(t):
            out = fn(t)
            if any(t is f for f in fixed) and (out.dtype != t.dtype or not out.is_contiguous()):
                return t.detach().to(out.device)
            return out

        return super()._apply(keep, recurse=False)

    def _load_from_state_dict(self, state_dict, prefix, metadata, strict, missing, unexpected, errors):
        for name in self.FIXED:
            own, t = getattr(self, name, None), state_dict.get(prefix + name)
            if own is None or own.dtype != torch.uint8 or not isinstance(t, torch.Tensor):
                continue
            # stored as float8_e4m3fn the codes are taken as they are, not converted as numbers
            if t.dtype == torch.float8_e4m3fn:
                state_dict[prefix + name] = t.view(torch.uint8)
            elif t.is_floating_point() and t.element_size() == 1:
                errors.append("%s%s: codes of type %s, expected uint8 or float8_e4m3fn"
                              % (prefix, name, t.dtype))
        super()._load_from_state_dict(state_dict, prefix, metadata, strict, missing, unexpected,
                                      errors)


class LinearBlockFp8(FixedTypes):
    """nn.Linear with a block-scaled e4m3 weight.

    Buffers (saved by ``state_dict``): ``CB`` uint8 [out, in] e4m3 codes, ``SCB`` fp32
    [ceil(out/128), ceil(in/128)], ``bias`` [out] or absent.  With ``has_16bit_weights`` the
    weight and the bias are parameters of type `dtype` instead, quantised by every forward, and
    the layer trains; without, it passes the gradient of its input.

    in_features must be a multiple of 16; out_features may be any number.  A cast of the model
    changes the type of weight and bias; codes and scales keep theirs.
    """

    FIXED = ("CB", "SCB")

    def __init__(self, in_features: int, out_features: int, bias: bool = True, device=None,
                 dtype: torch.dtype = torch.bfloat16, has_16bit_weights: bool = False):
        super().__init__()
        if in_features <= 0 or out_features <= 0 or in_features % 16 != 0:
            raise ValueError("in_features must be a positive multiple of 16 (row pitch of the "
                             "codes for TMA); out_features positive")
        if dtype not in DTYPES:
            raise TypeError("dtype must be torch.float16 or torch.bfloat16")
        self.in_features = in_features
        self.out_features = out_features
        self.has_16bit_weights = bool(has_16bit_weights)
        b = torch.zeros((out_features,), dtype=dtype, device=device) if bias else None
        if self.has_16bit_weights:
            self.weight = torch.nn.Parameter(
                torch.zeros((out_features, in_features), dtype=dtype, device=device))
            self.bias = None if b is None else torch.nn.Parameter(b)
        else:
            self.register_buffer("CB", torch.zeros((out_features, in_features),
                                                   dtype=torch.uint8, device=device))
            self.register_buffer("SCB", torch.ones(((out_features + 127) // 128,
                                                    (in_features + 127) // 128),
                                                   dtype=torch.float32, device=device))
            self.register_buffer("bias", b)

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear, has_16bit_weights: bool = False,
                    dtype: Optional[torch.dtype] = None) -> "LinearBlockFp8":
        """From an nn.Linear on a CUDA device.  dtype: by default the weight's, if it has 16
        bits, else bf16 (to which the weight is rounded before it is quantised)."""
        w = linear.weight
        if not w.is_cuda:
            raise ValueError("the weight must be on a CUDA device (it is quantised there)")
        dtype = dtype or (w.dtype if w.dtype in DTYPES else torch.bfloat16)
        m = cls(linear.in_features, linear.out_features, bias=linear.bias is not None,
                device=w.device, dtype=dtype, has_16bit_weights=has_16bit_weights)
        with torch.no_grad():
            if has_16bit_weights:
                m.weight.copy_(w.to(dtype))
            else:
                m.CB, m.SCB = quantize_weight_blocks(w.to(dtype))
            if linear.bias is not None:
                m.bias.copy_(linear.bias.to(dtype))
        return m

    @classmethod
    def from_codes(cls, codes: torch.Tensor, scales: torch.Tensor,
                   bias: Optional[torch.Tensor] = None,
                   dtype: torch.dtype = torch.bfloat16) -> "LinearBlockFp8":
        """From a stored weight: e4m3 codes [N, K] (float8_e4m3fn or uint8) and fp32 scales
        [ceil(N/128), ceil(K/128)]."""
        if codes.dim() != 2 or codes.dtype not in (torch.uint8, torch.float8_e4m3fn):
            raise ValueError("codes: a 2-D tensor of float8_e4m3fn or uint8 is required")
        N, K = codes.shape
        if tuple(scales.shape) != ((N + 127) // 128, (K + 127) // 128):
            raise ValueError("scales of shape %s, expected %s"
                             % (tuple(scales.shape), ((N + 127) // 128, (K + 127) // 128)))
        m = cls(K, N, bias=bias is not None, device=codes.device, dtype=dtype)
        m.CB.copy_(codes.view(torch.uint8))
        m.SCB.copy_(scales)
        if bias is not None:
            m.bias.copy_(bias.to(dtype))
        return m

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if self.bias is not None and x.dtype != self.bias.dtype:
            raise TypeError("input must be %s, the bias' type (got %s)" % (self.bias.dtype, x.dtype))
        if self.has_16bit_weights:
            return linear_block_fp8_train(x, self.weight, self.bias)
        return linear_block_fp8(x, self.CB, self.SCB, self.bias)

    def extra_repr(self) -> str:
        return ("in_features=%d, out_features=%d, bias=%s, has_16bit_weights=%s"
                % (self.in_features, self.out_features, self.bias is not None,
                   self.has_16bit_weights))


def replace_linear_with_block_fp8(model: torch.nn.Module, skip: Iterable[str] = ("lm_head",),
                                  has_16bit_weights: bool = False,
                                  dtype: Optional[torch.dtype] = None) -> torch.nn.Module:
    """Swap every nn.Linear of `model` (weights on a CUDA device) for a LinearBlockFp8, in
    place, except modules whose name (last path component) is in `skip`.  Returns `model`."""
    skip = set(skip)
    for name, child in list(model.named_children()):
        if name in skip:
            continue
        if isinstance(child, torch.nn.Linear):
            setattr(model, name, LinearBlockFp8.from_linear(child, has_16bit_weights, dtype))
        else:
            replace_linear_with_block_fp8(child, skip, has_16bit_weights, dtype)
    return model
