"""Derivatives that the block-scaled layers, routing and experts do not have, on the CPU: they are
refused, never left out of a sum.  The library's calls are replaced by ones that only fill the
buffers, so the front ends run without a GPU."""
import contextlib

import pytest
import torch
import torch.autograd.forward_ad as fwAD

from bit_matmul_decomposition_b200 import abi, block, experts

T, K, N, E, I, k = 4, 32, 16, 3, 16, 2
H = torch.bfloat16


@pytest.fixture
def filled(monkeypatch):
    """Every launch writes ones into its outputs."""
    def fill(*outputs):
        def fn(*args, **_):
            for i in outputs:
                if args[i] is not None:
                    args[i].fill_(1)
        return fn
    for name, outputs in (("i8_block_linear_forward", (4,)), ("i8_block_linear_backward", (4, 5, 6)),
                          ("i8_block_quantize_weight", (1, 2)), ("i8_route_experts", (8, 9)),
                          ("i8_route_experts_backward", (6,)), ("i8_experts_forward", (7, 8)),
                          ("i8_experts_backward", (8, 9))):
        monkeypatch.setattr(abi, name, fill(*outputs))
    for name in ("i8_block_linear_workspace_size", "i8_block_linear_backward_workspace_size",
                 "i8_experts_workspace_size", "i8_experts_backward_workspace_size"):
        monkeypatch.setattr(abi, name, lambda *a: 16)
    for m in (block, experts):
        monkeypatch.setattr(m, "_on", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(block, "quantize_weight_blocks",
                        lambda w: (torch.ones(w.shape, dtype=torch.uint8), torch.ones((1, 1))))


def _linear():
    return (torch.ones((T, K), dtype=H), torch.ones((N, K), dtype=torch.uint8), torch.ones((1, 1)), torch.ones((N,), dtype=H))


def _experts():
    return (torch.ones((T, K), dtype=H), torch.zeros((T, k), dtype=torch.int32), torch.ones((T, k)),
            torch.ones((E, 2, I, K), dtype=torch.uint8), torch.ones((E, 2, 1, 1)), torch.ones((E, K, I), dtype=torch.uint8),
            torch.ones((E, 1, 1)))


# ------------------------------------------------------------------ forward mode
@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("which", ["x", "scales", "bias"])
def test_linear_refuses_tangents(filled, which, grad):
    a = dict(zip(("x", "codes", "scales", "bias"), _linear()))
    with fwAD.dual_level(), torch.set_grad_enabled(grad):
        block.linear_block_fp8(**a)                        # no tangent: runs
        a[which] = fwAD.make_dual(a[which], torch.ones_like(a[which]))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            block.linear_block_fp8(**a)


@pytest.mark.parametrize("which", ["x", "weight", "bias"])
def test_training_linear_refuses_tangents(filled, which):
    x, _, _, b = _linear()
    a = dict(x=x, weight=torch.ones((N, K), dtype=H), bias=b)
    with fwAD.dual_level():
        block.linear_block_fp8_train(**a)
        a[which] = fwAD.make_dual(a[which], torch.ones_like(a[which]))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            block.linear_block_fp8_train(**a)


@pytest.mark.parametrize("which", [0, 2, 4, 6])            # x, weights, S13, S2
def test_experts_refuse_tangents(filled, which):
    a = list(_experts())
    with fwAD.dual_level():
        experts.experts_block_fp8(*a)
        a[which] = fwAD.make_dual(a[which], torch.ones_like(a[which]))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            experts.experts_block_fp8(*a)


@pytest.mark.parametrize("which", ["logits", "balance"])
def test_routing_refuses_tangents(which):
    a = dict(logits=torch.ones((T, E)), top_k=k, balance=torch.ones((E,)))
    with fwAD.dual_level():
        a[which] = fwAD.make_dual(a[which], torch.ones_like(a[which]))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            experts.route_experts(**a)
