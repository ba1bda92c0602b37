"""Linear8bitLt on the CPU: derivatives that it does not have are refused, and casts of a model leave
its codes and scales alone.  The library's calls are replaced by ones that only make the buffers."""
import contextlib

import pytest
import torch
import torch.autograd.forward_ad as fwAD

from bit_matmul_decomposition_b200 import abi, linear

T, K, N = 4, 32, 16
H = torch.float16


def _layer(monkeypatch, fp16_weights):
    m = linear.Linear8bitLt(K, N, has_fp16_weights=fp16_weights)
    monkeypatch.setattr(m, "_forward_kernel", lambda x: torch.ones((x.shape[0], N), dtype=H))
    monkeypatch.setattr(m, "_quantize", lambda w: None)
    monkeypatch.setattr(m, "dequantized_weight", lambda: torch.ones((N, K), dtype=H))
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    for name, at in (("i8_linear_backward_input", 2), ("i8_linear_backward_weight", 2), ("i8_bias_grad", 1)):
        monkeypatch.setattr(abi, name, lambda *a, at=at: a[at].fill_(1))
    return m


@pytest.mark.parametrize("fp16_weights", [True, False])
@pytest.mark.parametrize("grad", [True, False])
def test_tangents_are_refused(monkeypatch, fp16_weights, grad):
    m = _layer(monkeypatch, fp16_weights)
    x = torch.ones((T, K), dtype=H)
    with fwAD.dual_level(), torch.set_grad_enabled(grad):
        m(x)
        with pytest.raises(NotImplementedError, match="forward-mode"):
            m(fwAD.make_dual(x, torch.ones_like(x)))


@pytest.mark.parametrize("which", ["weight", "bias"])
def test_tangents_of_parameters_are_refused(monkeypatch, which):
    m = _layer(monkeypatch, True)
    x = torch.ones((T, K), dtype=H)
    with fwAD.dual_level():
        p = getattr(m, which).detach().clone()
        delattr(m, which)
        setattr(m, which, fwAD.make_dual(p, torch.ones_like(p)))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            m(x)


@pytest.mark.parametrize("fp16_weights", [True, False])
def test_second_derivatives_are_refused(monkeypatch, fp16_weights):
    m = _layer(monkeypatch, fp16_weights)
    x = torch.ones((T, K), dtype=H, requires_grad=True)
    if fp16_weights:
        for of, to in ((x, m.weight), (m.weight, x)):      # each gradient depends on the other operand
            first, = torch.autograd.grad(m(x).float().sum(), of, create_graph=True)
            with pytest.raises(NotImplementedError, match="second"):
                torch.autograd.grad(first.float().square().sum() + to.float().square().sum(), to)
        first, = torch.autograd.grad(m(x).float().sum(), m.bias, create_graph=True)
        assert not first.requires_grad
    y = m(x)
    gy = torch.ones_like(y).requires_grad_(True)
    first, = torch.autograd.grad(y, x, gy, create_graph=True)
    with pytest.raises(NotImplementedError, match="second"):
        torch.autograd.grad(first.float().square().sum() + gy.float().square().sum(), gy)


def test_create_graph_gives_the_same_gradients(monkeypatch):
    m = _layer(monkeypatch, True)
    x = torch.ones((T, K), dtype=H, requires_grad=True)
    wanted = (x, m.weight, m.bias)
    for a, b in zip(torch.autograd.grad(m(x).float().sum(), wanted),
                    torch.autograd.grad(m(x).float().sum(), wanted, create_graph=True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cast", [lambda m: m.half(), lambda m: m.to(torch.bfloat16), lambda m: m.half().float(),
                                  lambda m: m.type(torch.float16)])
@pytest.mark.parametrize("fp16_weights,code_format", [(False, "int8"), (False, "e4m3"), (True, "int8")])
def test_casts_leave_codes_and_scales(cast, fp16_weights, code_format):
    g = torch.Generator().manual_seed(2)
    m = linear.Linear8bitLt(K, N, has_fp16_weights=fp16_weights, code_format=code_format)
    m.CB.copy_(torch.randint(0, 127, (N, K), generator=g))
    m.SCB.copy_(torch.rand(N, generator=g))
    codes, scales = m.CB.clone(), m.SCB.clone()
    m = cast(torch.nn.Sequential(m))[0]
    assert m.CB.dtype == codes.dtype and torch.equal(m.CB, codes)
    assert m.SCB.dtype == torch.float32 and torch.equal(m.SCB, scales)
