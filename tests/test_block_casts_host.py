"""Casts of whole models, on the CPU: what has to stay fp32 (scales, balance, router) stays, bit for
bit, and the codes stay codes; the rest follows the cast."""
import copy

import pytest
import torch

from bit_matmul_decomposition_b200 import block, experts

KEPT = {"CB", "SCB", "CB13", "S13", "CB2", "S2", "balance", "gate"}


def _layer(kind):
    g = torch.Generator().manual_seed(5)
    if kind in ("frozen", "train"):
        m = block.LinearBlockFp8(144, 40, has_16bit_weights=kind == "train")
    elif kind == "experts":
        m = experts.ExpertsBlockFp8(3, 144, 32)
    else:
        m = experts.RoutedExperts(experts.ExpertsBlockFp8(3, 144, 32), 2, torch.randn(3, 144, generator=g), balance=True)
    for _, b in m.named_buffers():
        b.copy_(torch.randint(0, 127, b.shape, generator=g) if b.dtype == torch.uint8 else
                torch.rand(b.shape, generator=g) * 1e-5)          # scales that fp16 could not hold
    return torch.nn.Sequential(m, torch.nn.Linear(4, 4))


CASTS = {
    "bfloat16": lambda m: m.bfloat16(), "half": lambda m: m.half(), "to": lambda m: m.to(torch.bfloat16),
    "double": lambda m: m.double(), "type": lambda m: m.type(torch.float16),
    "device and type": lambda m: m.to("cpu", torch.float16),
    "there and back": lambda m: m.half().float(), "copy": lambda m: copy.deepcopy(m).half(),
}


@pytest.mark.parametrize("cast", list(CASTS))
@pytest.mark.parametrize("kind", ["frozen", "train", "experts", "routed"])
def test_casts_keep_scales_codes_and_router(kind, cast):
    m = _layer(kind)
    before = {n: t.detach().clone() for n, t in m[0].state_dict().items()}
    other = dict(m[0].named_parameters())
    m = CASTS[cast](m)
    after = m[0].state_dict()
    assert set(after) == set(before)
    for n, t in after.items():
        name = n.split(".")[-1]
        if name in KEPT:
            assert t.dtype == before[n].dtype and torch.equal(t, before[n]), n
    if cast != "copy":                                     # parameters keep their identity
        assert all(dict(m[0].named_parameters())[n] is p for n, p in other.items())
    if kind == "train":                                    # the 16-bit weight follows the cast
        want = {"there and back": torch.float32, "double": torch.float64, "bfloat16": torch.bfloat16, "to": torch.bfloat16}
        assert m[0].weight.dtype == want.get(cast, torch.float16) == m[0].bias.dtype == m[1].weight.dtype


def test_a_cast_keeps_the_routers_gradient():
    m = _layer("routed")
    r = m[0]
    r.gate.grad = torch.rand_like(r.gate) * 1e-6
    g = r.gate.grad.clone()
    m.half()
    assert r.gate.grad.dtype == torch.float32 and torch.equal(r.gate.grad, g) and r.gate.requires_grad


def test_moves_still_move():
    m = _layer("routed").to("meta")
    assert all(t.is_meta for t in (*m.parameters(), *m.buffers()))
    assert m[0].experts.S13.dtype == torch.float32
    m = m.half().to_empty(device="cpu")
    assert m[0].experts.S13.dtype == torch.float32 and not m[0].gate.is_meta and m[1].weight.dtype == torch.float16


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_router_logits_stay_fp32_under_autocast(monkeypatch, dtype):
    seen = {}

    def route(logits, *a, **kw):
        seen["logits"] = logits
        return torch.ones((*logits.shape[:-1], 2)), torch.zeros((*logits.shape[:-1], 2), dtype=torch.int32)
    monkeypatch.setattr(experts, "route_experts", route)
    monkeypatch.setattr(experts, "experts_block_fp8", lambda x, *a: x)
    r = _layer("routed")[0]
    x = torch.randn(5, 144, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    r(x)
    plain = seen["logits"]
    with torch.autocast("cpu", dtype=dtype):
        r(x)
        assert torch.is_autocast_enabled("cpu")
    assert seen["logits"].dtype == torch.float32 and torch.equal(seen["logits"], plain)
    seen["logits"].sum().backward()
    assert torch.equal(r.gate.grad, x.float().sum(0).expand(3, 144))


def test_a_memory_format_leaves_the_layout():
    """channels_last reorders 4-D tensors; the library takes codes and scales row by row."""
    m = _layer("experts")
    before = {n: t.clone() for n, t in m[0].state_dict().items()}
    for fmt in (torch.channels_last, torch.contiguous_format):
        m = m.to(torch.float16, memory_format=fmt)
        for n, t in m[0].state_dict().items():
            assert t.is_contiguous() and t.dtype == before[n].dtype and torch.equal(t, before[n]), n


@pytest.mark.parametrize("assign", [False, True])
@pytest.mark.parametrize("kind", ["frozen", "experts", "routed"])
def test_stored_float8_codes_load_as_codes(kind, assign):
    """A checkpoint's codes are float8_e4m3fn; copied into bytes as numbers, 1.5 would become 1."""
    m = _layer(kind)[0]
    state = m.state_dict()
    stored = {n: t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t.clone() for n, t in state.items()}
    want = {n: t.clone() for n, t in state.items()}
    fresh = _layer(kind)[0]
    for b in fresh.buffers():
        b.zero_()
    fresh.load_state_dict(stored, assign=assign)
    for n, t in fresh.state_dict().items():
        assert t.dtype == want[n].dtype and torch.equal(t, want[n]), n
    assert any(t.dtype == torch.float8_e4m3fn for t in stored.values())    # the caller's stay as they were


@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.float8_e4m3fnuz])
def test_other_8_bit_floats_do_not_load(dtype):
    m = _layer("frozen")[0]
    state = dict(m.state_dict())
    state["CB"] = torch.zeros(state["CB"].shape).to(dtype)
    with pytest.raises(RuntimeError, match="float8_e4m3fn"):
        m.load_state_dict(state)
