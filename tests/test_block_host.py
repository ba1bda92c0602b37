"""Host-side checks of the block-scaled calls, routing and experts (no GPU): the library refuses
bad sizes and pointers before it touches CUDA, the binding holds every tensor to its type and
size, and the front ends refuse what the kernels do not take."""
import math

import pytest
import torch

from bit_matmul_decomposition_b200 import abi, block, build, experts

INVALID = 1
F = 0x10000     # aligned, never dereferenced: validation rejects before any launch


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.load()


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(abi, "load", lambda *a, **k: r)
    monkeypatch.setattr(abi, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(abi, "_stream", lambda s: 0)
    return r


def _t(shape, dtype):
    return torch.zeros(shape, dtype=dtype)


# ------------------------------------------------------------------ the library
def test_workspace_sizes(lib):
    f, b = lib.i8_block_linear_workspace_size, lib.i8_block_linear_backward_workspace_size
    for size in (f, b):
        assert size(0, 64, 64) == 0 and size(4, 0, 64) == 0 and size(4, 64, 72) == 0
        assert size(4, 64, -16) == 0 and size(1 << 31, 64, 64) == 0
    assert f(2048, 16384, 4096) >= 2048 * 4096 + 32 * 2048 * 4
    assert f(1, 16384, 4096) >= 4096 + 32 * 4 + 2 * 148 * 16 * 128 * 4      # partial tiles
    assert b(300, 605, 1040) >= 2 * 300 * 608 + 300 * 1040
    for size in (lib.i8_experts_workspace_size, lib.i8_experts_backward_workspace_size):
        assert size(0, 128, 128, 4, 2) == 0 and size(4, 136, 128, 4, 2) == 0 and size(4, 128, 120, 4, 2) == 0
        assert size(4, 128, 128, 513, 2) == 0 and size(4, 128, 128, 4, 0) == 0 and size(4, 128, 128, 4, 33) == 0
        assert size(1 << 30, 128, 128, 4, 2) == 0                          # T * k past 32 bits
        assert size(4, 128, 128, 4, 2) > 0


def test_forward_refusals(lib):
    ws = lib.i8_block_linear_workspace_size(32, 64, 64)

    def call(**kw):
        a = dict(X=F, dt=1, T=32, K=64, CB=F, SCB=F, bias=None, N=64, Y=F, ws=F, n=ws)
        a.update(kw)
        return lib.i8_block_linear_forward(a["X"], a["dt"], a["T"], a["K"], a["CB"], a["SCB"], a["bias"], a["N"], a["Y"],
                                           a["ws"], a["n"], None)

    for name in ("X", "CB", "SCB", "Y", "ws"):
        assert call(**{name: None}) == INVALID and call(**{name: F + 8}) == INVALID
    assert call(bias=F + 2) == INVALID
    for kw in (dict(dt=2), dict(dt=-1), dict(T=0), dict(T=-1), dict(K=72), dict(K=0), dict(N=0), dict(N=1 << 31),
               dict(T=1 << 31), dict(n=ws - 1)):
        assert call(**kw) == INVALID


def test_backward_refusals(lib):
    ws = lib.i8_block_linear_backward_workspace_size(32, 64, 64)

    def call(**kw):
        a = dict(dY=F, X=F, dt=0, T=32, N=64, K=64, CB=F, SCB=F, dX=F, dW=F, db=F, ws=F, n=ws)
        a.update(kw)
        return lib.i8_block_linear_backward(a["dY"], a["X"], a["dt"], a["T"], a["N"], a["K"], a["CB"], a["SCB"], a["dX"],
                                            a["dW"], a["db"], a["ws"], a["n"], None)

    for kw in (dict(dY=None), dict(ws=None), dict(dX=None, dW=None, db=None), dict(CB=None), dict(SCB=None), dict(X=None),
               dict(dX=F + 4), dict(dW=F + 4), dict(db=F + 4), dict(X=F + 4), dict(dt=2), dict(K=8), dict(T=0), dict(N=0),
               dict(n=ws - 1)):
        assert call(**kw) == INVALID


def test_quantiser_refusals(lib):
    q, w = lib.i8_block_quantize_act, lib.i8_block_quantize_weight
    assert q(None, 0, 4, 64, F, F, None) == INVALID and q(F, 3, 4, 64, F, F, None) == INVALID
    assert q(F, 0, 4, 40, F, F, None) == INVALID and q(F, 0, 0, 64, F, F, None) == INVALID
    assert w(F, 0, 0, 64, 64, F, F, None) == INVALID and w(F, 0, 1, 64, 40, F, F, None) == INVALID
    assert w(F, 2, 1, 64, 64, F, F, None) == INVALID and w(F, 0, 1, 64, 64, F + 1, F, None) == INVALID
    assert w(F, 0, 1 << 30, 64, 1 << 20, F, F, None) == INVALID


def test_route_refusals(lib):
    def call(**kw):
        a = dict(x=F, dt=2, T=4, E=64, bal=None, score=0, g=8, tg=4, k=8, scale=1.0, w=F, i=F)
        a.update(kw)
        return lib.i8_route_experts(a["x"], a["dt"], a["T"], a["E"], a["bal"], a["score"], a["g"], a["tg"], a["k"], 1,
                                    a["scale"], a["w"], a["i"], None)

    for kw in (dict(x=None), dict(w=None), dict(i=None), dict(bal=F + 4), dict(dt=3), dict(T=0), dict(E=0), dict(E=513),
               dict(score=2), dict(g=0), dict(g=5), dict(g=64), dict(tg=0), dict(tg=9), dict(k=0), dict(k=33),
               dict(E=4, g=1, tg=1, k=5), dict(scale=math.nan)):
        assert call(**kw) == INVALID
    b = lib.i8_route_experts_backward
    assert b(F, 2, 4, 64, 0, 8, 1, 1.0, None, F, F, None) == INVALID
    assert b(F, 2, 4, 64, 0, 65, 1, 1.0, F, F, F, None) == INVALID
    assert b(F, 2, 4, 64, 0, 8, 1, 1.0, F, F, F + 4, None) == INVALID


def test_experts_refusals(lib):
    ws = lib.i8_experts_workspace_size(4, 128, 128, 8, 2)

    def call(**kw):
        a = dict(X=F, dt=1, T=4, K=128, i=F, w=F, k=2, c=F, s=F, c2=F, s2=F, E=8, I=128, Y=F, gu=None, ws=F, n=ws)
        a.update(kw)
        return lib.i8_experts_forward(a["X"], a["dt"], a["T"], a["K"], a["i"], a["w"], a["k"], a["c"], a["s"], a["c2"],
                                      a["s2"], a["E"], a["I"], a["Y"], a["gu"], a["ws"], a["n"], None)

    for name in ("X", "i", "w", "c", "s", "c2", "s2", "Y", "ws"):
        assert call(**{name: None}) == INVALID and call(**{name: F + 4}) == INVALID
    for kw in (dict(gu=F + 4), dict(dt=2), dict(T=0), dict(K=120), dict(I=24), dict(E=0), dict(E=513), dict(k=0),
               dict(k=33), dict(n=ws - 1)):
        assert call(**kw) == INVALID
    bws = lib.i8_experts_backward_workspace_size(4, 128, 128, 8, 2)
    b = lib.i8_experts_backward
    assert b(F, 1, 4, 128, F, F, 2, F, F, F, F, 8, 128, None, F, F, F, bws, None) == INVALID
    assert b(F, 1, 4, 128, F, F, 2, F, F, F, F, 8, 128, F, F, F, F, bws - 1, None) == INVALID


# ------------------------------------------------------------------ the binding
T, K, N, E, I, k = 5, 144, 40, 3, 160, 2
H = torch.bfloat16


def test_linear_binding_marshals_and_checks(rec):
    a = dict(X=_t((T, K), H), CB=_t((N, K), torch.uint8), SCB=_t((1, 2), torch.float32), bias=_t((N,), H), Y=_t((T, N), H),
             workspace=_t((99,), torch.uint8))
    abi.i8_block_linear_forward(**a)
    name, args = rec.calls[-1]
    assert name == "i8_block_linear_forward" and args[1:4] == (1, T, K) and args[7] == N and args[10] == 99
    for field, bad, err in (("X", _t((T, K), torch.float32), TypeError), ("X", _t((T * K,), H), ValueError),
                            ("CB", _t((N, K - 16), torch.uint8), ValueError), ("CB", _t((N, K), torch.int8), TypeError),
                            ("SCB", _t((1, 1), torch.float32), ValueError), ("SCB", _t((1, 2), H), TypeError),
                            ("bias", _t((N,), torch.float16), TypeError), ("bias", _t((N - 1,), H), ValueError),
                            ("Y", _t((T, N - 1), H), ValueError), ("Y", _t((T, N), torch.float16), TypeError)):
        with pytest.raises(err):
            abi.i8_block_linear_forward(**dict(a, **{field: bad}))
    assert len(rec.calls) == 1


def test_quantiser_binding(rec):
    abi.i8_block_quantize_act(_t((T, K), torch.float16), _t((T, K), torch.uint8), _t((2, T), torch.float32))
    assert rec.calls[-1][1][1:4] == (0, T, K)
    with pytest.raises(ValueError, match="SX"):
        abi.i8_block_quantize_act(_t((T, K), H), _t((T, K), torch.uint8), _t((2, T - 1), torch.float32))
    abi.i8_block_quantize_weight(_t((E, 2, I, K), H), _t((E, 2, I, K), torch.uint8), _t((E, 2, 2, 2), torch.float32))
    assert rec.calls[-1][1][1:5] == (1, 2 * E, I, K)
    with pytest.raises(ValueError, match="SCB"):
        abi.i8_block_quantize_weight(_t((I, K), H), _t((I, K), torch.uint8), _t((3,), torch.float32))
    with pytest.raises(TypeError, match="W"):
        abi.i8_block_quantize_weight(_t((I, K), torch.float32), _t((I, K), torch.uint8), _t((4,), torch.float32))


def test_backward_binding(rec):
    a = dict(dY=_t((T, N), H), X=_t((T, K), H), CB=_t((N, K), torch.uint8), SCB=_t((2,), torch.float32), dX=_t((T, K), H),
             dW=_t((N, K), H), db=_t((N,), H), workspace=_t((9,), torch.uint8))
    abi.i8_block_linear_backward(**a)
    assert rec.calls[-1][1][3:6] == (T, N, K)
    abi.i8_block_linear_backward(**dict(a, dX=None, CB=None, SCB=None))
    abi.i8_block_linear_backward(**dict(a, dW=None, X=None))
    abi.i8_block_linear_backward(**dict(a, dW=None, dX=None, X=None, CB=None, SCB=None))
    n = len(rec.calls)
    for kw in (dict(X=_t((T + 1, K), H)), dict(X=_t((T, K + 16), H)), dict(CB=_t((N + 1, K), torch.uint8)),
               dict(dX=_t((T - 1, K), H)), dict(dW=_t((N, K - 1), H)), dict(db=_t((N - 1,), H)), dict(X=None), dict(CB=None)):
        with pytest.raises(ValueError):
            abi.i8_block_linear_backward(**dict(a, **kw))
    with pytest.raises(TypeError):
        abi.i8_block_linear_backward(**dict(a, dW=_t((N, K), torch.float16)))
    assert len(rec.calls) == n


def test_route_and_experts_binding(rec):
    x = _t((T, 8), torch.float32)
    abi.i8_route_experts(x, None, "sigmoid", 2, 1, k, True, 1.0, _t((T, k), torch.float32), _t((T, k), torch.int32))
    assert rec.calls[-1][1][1:4] == (2, T, 8) and rec.calls[-1][1][5] == 1
    with pytest.raises(ValueError, match="idx"):
        abi.i8_route_experts(x, None, "sigmoid", 2, 1, k, True, 1.0, _t((T, k), torch.float32), _t((T, 1), torch.int32))
    with pytest.raises(TypeError, match="logits"):
        abi.i8_route_experts(x.double(), None, "softmax", 1, 1, k, True, 1.0, _t((T, k), torch.float32), _t((T, k), torch.int32))
    a = dict(X=_t((T, K), H), idx=_t((T, k), torch.int32), weights=_t((T, k), torch.float32),
             CB13=_t((E, 2, I, K), torch.uint8), S13=_t((E, 2, 2, 2), torch.float32), CB2=_t((E, K, I), torch.uint8),
             S2=_t((E, 2, 2), torch.float32), Y=_t((T, K), H), GU=None, workspace=_t((9,), torch.uint8))
    abi.i8_experts_forward(**a)
    assert rec.calls[-1][1][2:4] == (T, K) and rec.calls[-1][1][6] == k and rec.calls[-1][1][11:13] == (E, I)
    n = len(rec.calls)
    for kw in (dict(CB13=_t((E, 2, I, K - 16), torch.uint8)), dict(CB13=_t((E, 1, I, K), torch.uint8)),
               dict(CB2=_t((E, I, K), torch.uint8)), dict(S13=_t((E, 2, 2, 1), torch.float32)), dict(S2=_t((E, 2, 1), torch.float32)),
               dict(weights=_t((T - 1, k), torch.float32)), dict(Y=_t((T, K - 1), H)), dict(GU=_t((T, 2, I), torch.float32))):
        with pytest.raises(ValueError):
            abi.i8_experts_forward(**dict(a, **kw))
    with pytest.raises(TypeError):
        abi.i8_experts_forward(**dict(a, idx=_t((T, k), torch.int64)))
    assert len(rec.calls) == n


# ------------------------------------------------------------------ the front ends
def test_modules_refuse_what_the_kernels_do_not_take():
    with pytest.raises(ValueError):
        block.LinearBlockFp8(72, 64)
    with pytest.raises(ValueError):
        block.LinearBlockFp8(64, 0)
    with pytest.raises(TypeError):
        block.LinearBlockFp8(64, 64, dtype=torch.float32)
    with pytest.raises(ValueError, match="CUDA"):
        block.LinearBlockFp8.from_linear(torch.nn.Linear(64, 64))
    with pytest.raises(ValueError):
        block.LinearBlockFp8.from_codes(_t((130, 64), torch.uint8), _t((1, 1), torch.float32))
    m = block.LinearBlockFp8(64, 32)
    with pytest.raises(TypeError):
        m(_t((4, 64), torch.float32))
    with pytest.raises(TypeError):
        m(_t((4, 64), torch.float16))                      # the bias is bf16
    with pytest.raises(ValueError):
        m(_t((4, 80), H))
    with pytest.raises(TypeError):
        block.linear_block_fp8_train(_t((4, 64), H), _t((32, 64), torch.float16))
    with pytest.raises(ValueError):
        experts.ExpertsBlockFp8(513, 64, 64)
    with pytest.raises(ValueError):
        experts.ExpertsBlockFp8(4, 64, 72)
    with pytest.raises(ValueError):
        experts.ExpertsBlockFp8.from_weights(_t((2, 2, 32, 64), H), _t((2, 32, 64), H))
    with pytest.raises(ValueError, match="bias"):
        experts.ExpertsBlockFp8.from_linears(*([torch.nn.Linear(16, 16)] for _ in range(3)))


def test_experts_front_end_checks_shapes_and_types():
    c = (_t((3, 2, 32, 64), torch.uint8), _t((3, 2, 1, 1), torch.float32), _t((3, 64, 32), torch.uint8), _t((3, 1, 1), torch.float32))
    x, i, w = _t((4, 64), H), _t((4, 2), torch.int32), _t((4, 2), torch.float32)
    for bad in ((x.float(), i, w), (x, i.long(), w), (x, i, w.half())):
        with pytest.raises(TypeError):
            experts.experts_block_fp8(*bad, *c)
    for bad in ((x[:, :48], i, w), (x, i[:3], w), (x, i, w[:, :1]), (x, _t((4, 33), torch.int32), _t((4, 33), torch.float32))):
        with pytest.raises(ValueError):
            experts.experts_block_fp8(*bad, *c)


def test_route_front_end_checks(monkeypatch):
    with pytest.raises(ValueError, match="CUDA"):
        experts.route_experts(_t((4, 8), torch.float32), 2)
    with pytest.raises(ValueError, match="score"):
        experts.route_experts(_t((4, 8), torch.float32), 2, score="tanh")
