"""The block-scaled modules inside a user's model, on the GPU: casts, autocast, gradients under
create_graph, weights that a program casts itself, capture of a step whose input is computed."""
import pytest
import torch

from bit_matmul_decomposition_b200 import abi
from bit_matmul_decomposition_b200 import block as B
from bit_matmul_decomposition_b200 import experts as X

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    abi.load()
    yield
    torch.cuda.synchronize()


@pytest.fixture(autouse=True)
def _status():
    yield
    st = abi.i8_sync_status()
    assert st == 0, abi.STATUS.get(st, st)


def _model(dtype=torch.bfloat16, E=6, K=144, I=128):
    g = torch.Generator(device=DEV).manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV) * 0.06  # noqa: E731
    lin = torch.nn.Linear(K, K).to(DEV, dtype)
    with torch.no_grad():
        lin.weight.copy_(rand(K, K))
        lin.bias.copy_(rand(K))
    routed = X.RoutedExperts(X.ExpertsBlockFp8.from_weights(rand(E, 2, I, K).to(dtype), rand(E, K, I).to(dtype)), 2,
                             10 * rand(E, K), balance=True, score="sigmoid", n_groups=3, top_groups=2)
    routed.balance.copy_(0.1 * rand(E))
    return torch.nn.Sequential(B.LinearBlockFp8.from_linear(lin), routed), g


@pytest.mark.parametrize("T", [3, 300])
def test_a_cast_model_gives_the_same_outputs(T):
    m, g = _model()
    x = torch.randn(T, 144, generator=g, device=DEV).to(torch.bfloat16)
    m[0].bias.copy_(torch.randint(-9, 10, (144,), generator=g, device=DEV) / 64)   # in any 16-bit type
    want = m(x)
    assert torch.equal(m.to(torch.bfloat16)(x), want)
    y = m.half()(x.half())
    assert y.dtype == torch.float16 and torch.isfinite(y).all()
    assert torch.equal(m.float().double().bfloat16()(x), want)


@pytest.mark.parametrize("T", [3, 300])
def test_autocast_chooses_the_same_experts(T):
    m, g = _model()
    x = torch.randn(T, 144, generator=g, device=DEV).to(torch.bfloat16).requires_grad_(True)
    dy = torch.randn(T, 144, generator=g, device=DEV).to(torch.bfloat16)
    wanted = (x, m[1].gate)
    want = torch.autograd.grad(m(x), wanted, dy)
    plain = m(x)
    with torch.autocast("cuda", dtype=torch.bfloat16):
        y = m(x)
    assert torch.equal(y, plain)
    for a, b in zip(torch.autograd.grad(y, wanted, dy), want):
        assert a.dtype == b.dtype and torch.equal(a, b)


def test_gradients_under_create_graph():
    m, g = _model()
    x = torch.randn(40, 144, generator=g, device=DEV).to(torch.bfloat16).requires_grad_(True)
    wanted = (x, m[1].gate)
    want = torch.autograd.grad(m(x).float().square().sum(), wanted)
    got = torch.autograd.grad(m(x).float().square().sum(), wanted, create_graph=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    with pytest.raises(NotImplementedError, match="second"):
        (got[1].square().sum() + m[1].gate.square().sum()).backward()


def test_a_weight_that_the_program_casts():
    """An fp32 master weight, rounded by the program on the way in."""
    T, K, N = 70, 144, 200
    g = torch.Generator(device=DEV).manual_seed(3)
    master = torch.randn(N, K, generator=g, device=DEV).requires_grad_(True)
    x = torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16).requires_grad_(True)
    dy = torch.randn(T, N, generator=g, device=DEV).to(torch.bfloat16)
    y = B.linear_block_fp8_train(x, master.to(torch.bfloat16))
    gx, gm = torch.autograd.grad(y, (x, master), dy)
    w = master.detach().to(torch.bfloat16).requires_grad_(True)
    z = B.linear_block_fp8_train(x, w)
    hx, hw = torch.autograd.grad(z, (x, w), dy)
    assert torch.equal(y, z) and torch.equal(gx, hx) and torch.equal(gm, hw.float())


@pytest.mark.parametrize("T", [3, 300])
def test_a_step_with_computed_inputs_captured(T):
    m, g = _model()
    x = torch.randn(T, 144, generator=g, device=DEV).to(torch.bfloat16).requires_grad_(True)
    dy = torch.randn(T, 144, generator=g, device=DEV).to(torch.bfloat16)
    wanted = (x, m[1].gate)

    def step():
        y = m(x * 1.0)                                     # inputs that are no leaves
        return [y.detach(), *torch.autograd.grad(y, wanted, dy)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.no_grad():
        x.copy_(torch.randn(T, 144, generator=g, device=DEV))
    graph.replay()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)
