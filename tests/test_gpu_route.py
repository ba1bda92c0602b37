"""Routing of tokens to experts on the GPU, against the token-by-token 64-bit reference."""
import math

import pytest
import torch

from bit_matmul_decomposition_b200 import abi
from bit_matmul_decomposition_b200.experts import route_experts
from tests import block_ref as R

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


def _logits(T, E, dtype, seed=0, masked=False):
    g = torch.Generator().manual_seed(seed)
    x = (2 * torch.randn(T, E, generator=g)).to(dtype)
    if masked:
        x[torch.rand(T, E, generator=g) < 0.4] = -math.inf
        x[::3] = -math.inf
    return x


def _weights_bound(ref, scale):
    """A score, its sum and their quotient in 64 bits; one rounding to fp32, and the product
    with `scale` (which fp32 holds)."""
    return 2.0 ** -24 * ref.abs() * 1.001 + 1e-45


CASES = [  # T, E, k, n_groups, top_groups
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (3, 8, 2, 1, 1), (5, 33, 5, 1, 1), (130, 64, 6, 1, 1), (50, 60, 4, 4, 2),
    (17, 512, 32, 32, 3), (9, 384, 8, 1, 1), (40, 24, 24, 8, 8), (33, 160, 6, 32, 5), (12, 40, 8, 8, 1),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype,masked,bal,renorm", [
    (torch.float32, False, True, True), (torch.bfloat16, True, False, True), (torch.float16, True, True, False)])
@pytest.mark.parametrize("T,E,k,n_groups,top_groups", CASES)
def test_choice_weights_and_gradient(T, E, k, n_groups, top_groups, dtype, masked, bal, renorm, score):
    x = _logits(T, E, dtype, T + E, masked)
    balance = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E)) if bal else None
    scale = 2.5 if bal else 1.0
    xd = x.to(DEV).requires_grad_(True)
    w, idx = route_experts(xd, k, None if balance is None else balance.to(DEV), score=score, n_groups=n_groups,
                           top_groups=top_groups, renormalize=renorm, scale=scale)
    rw, ri, P = R.route(x, k, balance, score, n_groups, top_groups, renorm, scale)
    assert torch.equal(idx.cpu(), ri)
    R.check(w, rw, _weights_bound(rw, scale), "weights")
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(7))
    w.backward(dw.to(DEV))
    ref = R.route_grad(P, ri, dw, score, renorm, scale)
    # one rounding to the logits' type; what cancels before it is 64-bit
    bound = R.half_step(dtype) * ref.abs() * 1.001 + 1e-13 * scale + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    R.check(xd.grad, ref, bound, "dlogits")


def test_equal_scores_take_the_lower_index():
    x = torch.zeros(3, 40, dtype=torch.bfloat16)
    x[1, 5:9] = 1.0
    x[2, 30:] = 100.0                                      # sigmoid: all 1 in fp32, and 1 - 4e-44 in 64 bits
    for score in ("softmax", "sigmoid"):
        w, idx = route_experts(x.to(DEV), 6, score=score)
        assert idx[0].tolist() == [0, 1, 2, 3, 4, 5]
        assert idx[1].tolist() == [5, 6, 7, 8, 0, 1]
        assert idx[2].tolist() == [30, 31, 32, 33, 34, 35]
        w, idx = route_experts(x.to(DEV), 6, score=score, n_groups=4, top_groups=2)
        assert idx[0].tolist() == [0, 1, 2, 3, 4, 5]


def test_scores_closer_than_fp32():
    """Two sigmoids that fp32 rounds to the same number keep their order."""
    x = torch.full((1, 8), -30.0)
    x[0, 2], x[0, 6] = 17.0, 17.5
    assert float(torch.sigmoid(x[0, 2])) == float(torch.sigmoid(x[0, 6]))
    w, idx = route_experts(x.to(DEV), 2, score="sigmoid")
    assert idx[0].tolist() == [6, 2]


def test_masked_rows_nan_and_infinity():
    x = _logits(6, 20, torch.float32, 3)
    x[0] = -math.inf
    x[1, 3:] = -math.inf
    x[2, 7] = math.nan
    x[3, 5] = math.inf
    for score in ("softmax", "sigmoid"):
        w, idx = route_experts(x.to(DEV), 5, score=score)
        assert (idx[0] == -1).all() and (w[0] == 0).all()
        assert (idx[1, 3:] == -1).all() and (w[1, 3:] == 0).all() and (idx[1, :3] >= 0).all()
        assert abs(float(w[1].sum()) - 1) < 1e-6
        assert torch.isnan(w[2]).all() and not (idx[2] == 7).any() and (idx[2] >= 0).all()
        assert idx[3, 0] == 5
        assert torch.isnan(w[3]).all() if score == "softmax" else torch.isfinite(w[3]).all()
        assert torch.isfinite(w[4:]).all()


def test_gradient_against_differences():
    x = _logits(4, 16, torch.float32, 9)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            dw = torch.randn(4, 3, generator=torch.Generator().manual_seed(1))
            xd = x.to(DEV).requires_grad_(True)
            w, idx = route_experts(xd, 3, score=score, renormalize=renorm)
            w.backward(dw.to(DEV))
            h = 1e-3                                       # central differences: error about h^2 times the third derivative
            for t, e in ((0, int(idx[0, 0])), (1, int(idx[1, 2])), (2, 5), (3, int(idx[3, 1]))):
                up, down = x.double(), x.double()
                up[t, e] += h
                down[t, e] -= h
                fu, iu, _ = R.route(up, 3, None, score, 1, 1, renorm, 1.0)
                fd, i0, _ = R.route(down, 3, None, score, 1, 1, renorm, 1.0)
                assert torch.equal(iu, i0)
                slope = float(((fu - fd) * dw).sum()) / (2 * h)
                assert abs(float(xd.grad[t, e]) - slope) < 1e-5


def test_strides_shapes_streams_and_capture():
    x = _logits(24, 64, torch.bfloat16, 4)
    rw, ri, _ = R.route(x, 4, None, "softmax", 1, 1, True, 1.0)
    wide = torch.zeros(24, 128, dtype=torch.bfloat16, device=DEV)
    wide[:, ::2] = x.to(DEV)
    w, idx = route_experts(wide[:, ::2].view(2, 12, 64), 4)
    assert w.shape == (2, 12, 4) and torch.equal(idx.view(24, 4).cpu(), ri)
    assert route_experts(x[:0].to(DEV), 4)[1].shape == (0, 4)
    xd = x.to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        w2, i2 = route_experts(xd, 4)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(i2.cpu(), ri) and torch.equal(w2, w.view(24, 4))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w3, i3 = route_experts(xd, 4)
    other = _logits(24, 64, torch.bfloat16, 5)
    xd.copy_(other)
    g.replay()
    assert torch.equal(i3.cpu(), R.route(other, 4, None, "softmax", 1, 1, True, 1.0)[1])


def test_more_than_2_31_logits():
    T, E = 4200000, 512
    x = torch.empty((T, E), dtype=torch.bfloat16, device=DEV)
    for i in range(0, T, 420000):
        x[i:i + 420000] = torch.randn(420000, E, device=DEV)
    x[-100:] = x[:100]
    w, idx = route_experts(x, 4, score="sigmoid")
    assert torch.equal(w[-100:], w[:100]) and torch.equal(idx[-100:], idx[:100])
    rw, ri, _ = R.route(x[-3:].cpu(), 4, None, "sigmoid", 1, 1, True, 1.0)
    assert torch.equal(idx[-3:].cpu(), ri)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_far_out_take_the_exact_scores(score):
    """Saturated sigmoids and scores that underflow: equal scores, so the lower index."""
    x = torch.full((4, 70), -3.0)
    x[0, 60], x[0, 10], x[0, 33] = 50.0, 40.0, 45.0        # sigmoid: all 1 in 64 bits
    x[1] = -1000.0
    x[1, 50], x[1, 3] = 0.0, -900.0                        # softmax: 0 but for one; sigmoid 0
    x[2, :] = torch.arange(70) * 0.1
    x[3, 40:] = -math.inf
    for groups, top in ((1, 1), (7, 3)):
        w, idx = route_experts(x.to(DEV), 5, score=score, n_groups=groups, top_groups=top)
        rw, ri, _ = R.route(x, 5, None, score, groups, top, True, 1.0)
        assert torch.equal(idx.cpu(), ri)
        R.check(w, rw, _weights_bound(rw, 1.0))
