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


# ------------------------------------------------------------------ second derivatives
def _calls():
    """Name: (call, its differentiable inputs, which inputs' gradients each gradient depends on,
    besides the gradient of the output)."""
    x, codes, scales, b = _linear()
    w = torch.ones((N, K), dtype=H)
    ex = _experts()
    logits = torch.ones((T, E))
    return {
        "linear": (lambda x, b: block.linear_block_fp8(x, codes, scales, b), (x, b), ((), ())),
        "train": (block.linear_block_fp8_train, (x, w, b), ((1,), (0,), ())),
        "route": (lambda v: experts._RouteFn.apply(v, None, "softmax", 1, 1, k, True, 1.0)[0], (logits,), ((0,),)),
        "experts": (lambda x, w: experts.experts_block_fp8(x, ex[1], w, *ex[3:]), (ex[0], ex[2]), ((0, 1), (0,))),
    }


@pytest.mark.parametrize("leaf", [True, False])
@pytest.mark.parametrize("name", ["linear", "train", "route", "experts"])
def test_second_derivatives_are_refused(filled, name, leaf):
    call, inputs, deps = _calls()[name]
    for i, needs in enumerate(deps):
        for other in range(len(inputs)):
            # the gradient of input i, differentiated again with respect to input `other`; the
            # loss reaches `other` by a second way, so that a lost term would raise nothing
            roots = [v.clone().requires_grad_(True) for v in inputs]
            args = roots if leaf else [v * 1 for v in roots]
            y = call(*args)
            first, = torch.autograd.grad(y.float().sum(), args[i], create_graph=True)
            loss = first.float().square().sum() + sum(v.float().square().sum() for v in roots)
            if other in needs:
                with pytest.raises(NotImplementedError, match="second"):
                    torch.autograd.grad(loss, roots[other])
            else:                                          # does not depend on it: nothing is lost
                torch.autograd.grad(loss, roots[other])
        # through the gradient of the output, on which every gradient depends
        roots = [v.clone().requires_grad_(True) for v in inputs]
        y = call(*roots)
        gy = torch.ones_like(y).requires_grad_(True)
        first, = torch.autograd.grad(y, roots[i], gy, create_graph=True)
        with pytest.raises(NotImplementedError, match="second"):
            torch.autograd.grad(first.float().square().sum() + gy.float().square().sum(), gy)


def test_first_derivatives_under_create_graph(filled):
    """Gradients taken with create_graph are the same, and may be used where nothing is
    differentiated again."""
    for name, (call, inputs, _) in _calls().items():
        roots = [v.clone().requires_grad_(True) for v in inputs]
        once = torch.autograd.grad(call(*roots).float().sum(), roots)
        again = torch.autograd.grad(call(*roots).float().sum(), roots, create_graph=True)
        assert all(torch.equal(a, b) for a, b in zip(once, again)), name
        call(*roots).float().sum().backward(create_graph=True)
        assert all(v.grad is not None for v in roots)


def test_frozen_inputs_carry_no_second_derivative(filled):
    """With a constant gradient of the output the frozen layer's dx is a constant."""
    x, codes, scales, b = _linear()
    x.requires_grad_(True)
    gx, = torch.autograd.grad(block.linear_block_fp8(x, codes, scales, b).float().sum(), x, create_graph=True)
    assert not gx.requires_grad
    w = torch.ones((N, K), dtype=H)
    gx, = torch.autograd.grad(block.linear_block_fp8_train(x, w, b).float().sum(), x, create_graph=True)
    assert not gx.requires_grad
