"""Experts with block-scaled weights on the GPU against the 64-bit reference.

Tolerance.  h is quantised between the products, so a difference of fp32 rounding size in h moves
those of its codes that lie at a rounding border by one e4m3 step (at most 2^-3 of the value).
With d the relative error of h's elements ((blocks + 40) 2^-23 times the ratio of the sum of
magnitudes to the value, and 2^-20 for the activation), the share of codes at a border is about
d / 2^-4, and each adds up to 2^-3 |h w2|: an output's error from it stays under
2^-3 max |h w2| times the few codes that move.  The tests bound an element by its half step, the
product's own bound, and FLIPS codes moved by 2^-3 of the largest term of its sum.
"""
import pytest
import torch

from bit_matmul_decomposition_b200 import abi
from bit_matmul_decomposition_b200 import block as B
from bit_matmul_decomposition_b200 import experts as X
from tests import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
FLIPS = 2


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


def _case(T, E, k, K, I, dtype, seed=0, none=0.15, skew=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g).to(dtype)
    x[:, ::37] *= 8
    w13 = (torch.randn(E, 2, I, K, generator=g) * 0.06).to(dtype)
    w2 = (torch.randn(E, K, I, generator=g) * 0.06).to(dtype)
    pop = torch.randn(T, E, generator=g) + skew * torch.randn(E, generator=g)
    idx = pop.topk(min(k, E), dim=1).indices.to(torch.int32)
    if k > E:
        idx = torch.cat([idx, idx[:, :k - E]], dim=1)
    idx[torch.rand(T, k, generator=g) < none] = -1
    w = torch.rand(T, k, generator=g)
    dy = (torch.randn(T, K, generator=g) * 0.1).to(dtype)
    return x, w13, w2, idx, w, dy


def _codes(w13, w2):
    CB13, S13 = B.quantize_weight_blocks(w13.to(DEV))
    CB2, S2 = B.quantize_weight_blocks(w2.to(DEV))
    E = w13.shape[0]
    W1 = [R.codes_value(CB13[e, 0], S13[e, 0]) for e in range(E)]
    W3 = [R.codes_value(CB13[e, 1], S13[e, 1]) for e in range(E)]
    W2 = [R.codes_value(CB2[e], S2[e]) for e in range(E)]
    return (CB13, S13, CB2, S2), W1, W3, W2


def _bounds(x, idx, w, W1, W3, W2, dy, y, dx, dw, dtype):
    """Allowed errors of y, dx and dw, from the magnitudes of the terms."""
    T, K = x.shape
    I = W1[0].shape[0]
    xq, dyq = R.rows_value(x), R.rows_value(dy)
    by, bx, bw = torch.zeros_like(y), torch.zeros_like(y), torch.zeros_like(dw)
    fk, fi = (-(-K // 128) + 40) * 2.0 ** -23, (-(-I // 128) + 40) * 2.0 ** -23
    for e in range(len(W1)):
        for t, j in torch.nonzero(idx == e).tolist():
            g, u = W1[e] @ xq[t], W3[e] @ xq[t]
            eg, eu = fk * (W1[e].abs() @ xq[t].abs()), fk * (W3[e].abs() @ xq[t].abs())
            sg = torch.sigmoid(g)
            h = g * sg * u
            # |silu'| <= 1.1, the activation a few steps of fp32
            eh = 1.1 * eg * u.abs() + (g * sg).abs() * eu + 2.0 ** -20 * h.abs()
            wt = float(w[t, j])
            term = (W2[e].abs() * (h.abs() + eh)[None])
            by[t] += wt * (fi * term.sum(1) + (W2[e].abs() * eh[None]).sum(1) + FLIPS * 2.0 ** -3 * term.max(1).values)
            dh = dyq[t] @ W2[e]
            ed = fk * (dyq[t].abs() @ W2[e].abs())
            bw[t, j] = (ed * h.abs() + dh.abs() * eh).sum() + (I + 40) * 2.0 ** -24 * (dh * h).abs().sum()
            ds = sg * (1 + g * (1 - sg))                   # its derivative is at most 0.5
            dg, du = wt * dh * u * ds, wt * dh * g * sg
            edg = wt * (ed * (u * ds).abs() + dh.abs() * (eu * 1.1 + u.abs() * 0.5 * eg)) + 2.0 ** -20 * (wt * dh * u).abs()
            edu = wt * (ed * (g * sg).abs() + dh.abs() * 1.1 * eg) + 2.0 ** -20 * du.abs()
            for v, ev, W in ((dg, edg, W1[e]), (du, edu, W3[e])):
                term = W.abs() * (v.abs() + ev)[:, None]
                bx[t] += 2 * fi * term.sum(0) + (W.abs() * ev[:, None]).sum(0) + FLIPS * 2.0 ** -3 * term.max(0).values
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    hs = R.half_step(dtype) * 1.01
    return by + hs * (y.abs() + by) + tiny, bx + hs * (dx.abs() + bx) + tiny, bw + 2.0 ** -24 * dw.abs() + 1e-30


CASES = [  # T, E, k, K, I
    (1, 4, 2, 256, 128), (1, 1, 1, 16, 16), (2, 8, 3, 144, 272), (7, 3, 5, 64, 144), (40, 6, 2, 256, 208),
    (33, 2, 2, 128, 128), (150, 3, 2, 272, 144), (300, 2, 2, 256, 160), (260, 1, 1, 128, 256),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,K,I", CASES)
def test_forward_and_gradients(T, E, k, K, I, dtype):
    x, w13, w2, idx, w, dy = _case(T, E, k, K, I, dtype, seed=T + E)
    codes, W1, W3, W2 = _codes(w13, w2)
    y, dx, dw = R.experts(x, idx, w, W1, W3, W2, dy)
    by, bx, bw = _bounds(x, idx, w, W1, W3, W2, dy, y, dx, dw, dtype)
    with torch.no_grad():
        R.check(X.experts_block_fp8(x.to(DEV), idx.to(DEV), w.to(DEV), *codes), y, by, "y without gradients")
    xd, wd = x.to(DEV).requires_grad_(True), w.to(DEV).requires_grad_(True)
    out = X.experts_block_fp8(xd, idx.to(DEV), wd, *codes)
    out.backward(dy.to(DEV))
    R.check(out, y, by, "y")
    R.check(xd.grad, dx, bx, "dx")
    R.check(wd.grad, dw, bw, "dw")


def test_all_tokens_to_one_expert_and_none_at_all():
    x, w13, w2, idx, w, dy = _case(90, 5, 2, 128, 144, torch.bfloat16)
    codes, W1, W3, W2 = _codes(w13, w2)
    idx[:] = 3                                             # twice the same expert
    y, dx, dw = R.experts(x, idx, w, W1, W3, W2, dy)
    by, bx, bw = _bounds(x, idx, w, W1, W3, W2, dy, y, dx, dw, torch.bfloat16)
    xd, wd = x.to(DEV).requires_grad_(True), w.to(DEV).requires_grad_(True)
    out = X.experts_block_fp8(xd, idx.to(DEV), wd, *codes)
    out.backward(dy.to(DEV))
    R.check(out, y, by)
    R.check(xd.grad, dx, bx)
    R.check(wd.grad, dw, bw)
    idx[:] = -1
    xd, wd = x.to(DEV).requires_grad_(True), w.to(DEV).requires_grad_(True)
    out = X.experts_block_fp8(xd, idx.to(DEV), wd, *codes)
    out.backward(dy.to(DEV))
    assert (out == 0).all() and (xd.grad == 0).all() and (wd.grad == 0).all()


@pytest.mark.parametrize("T", [3, 400])
def test_not_finite_tokens_stay_alone(T):
    x, w13, w2, idx, w, dy = _case(T, 2, 1, 128, 128, torch.bfloat16, none=0.0)
    codes, W1, W3, W2 = _codes(w13, w2)
    clean = X.experts_block_fp8(x.to(DEV), idx.to(DEV), w.to(DEV), *codes)
    x[1, 5] = float("nan")
    x[2, 9] = float("inf")
    w[0] = float("nan")
    idx[0] = -1                                            # the weight of no expert is not read
    y = X.experts_block_fp8(x.to(DEV), idx.to(DEV), w.to(DEV), *codes)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all() and (y[0] == 0).all()
    assert torch.equal(y[3:], clean[3:])


def test_an_index_past_the_experts_is_left_out_and_reported():
    x, w13, w2, idx, w, dy = _case(20, 4, 2, 128, 128, torch.bfloat16, none=0.0)
    codes, *_ = _codes(w13, w2)
    bad = idx.clone()
    bad[5, 1] = 4
    gone = idx.clone()
    gone[5, 1] = -1
    y = X.experts_block_fp8(x.to(DEV), bad.to(DEV), w.to(DEV), *codes)
    assert abi.i8_sync_status() == 5                       # I8_ERR_DEVICE, and cleared
    assert torch.equal(y, X.experts_block_fp8(x.to(DEV), gone.to(DEV), w.to(DEV), *codes))


@pytest.mark.parametrize("T", [1, 30, 300])
def test_repeated_streamed_and_captured(T):
    x, w13, w2, idx, w, dy = _case(T, 4, 2, 256, 144, torch.bfloat16)
    codes, W1, W3, W2 = _codes(w13, w2)
    xd, idd, wd = x.to(DEV), idx.to(DEV), w.to(DEV)
    first = X.experts_block_fp8(xd, idd, wd, *codes)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = [X.experts_block_fp8(xd, idd, wd, *codes) for _ in range(3)]
    here = [X.experts_block_fp8(xd, idd, wd, *codes) for _ in range(3)]
    torch.cuda.synchronize()
    for y in (*other, *here):
        assert torch.equal(y, first)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(X.experts_block_fp8(xd, idd, wd, *codes))
        graphs.append(g)
    x2, _, _, idx2, w2_, _ = _case(T, 4, 2, 256, 144, torch.bfloat16, seed=99)
    xd.copy_(x2)
    idd.copy_(idx2)
    wd.copy_(w2_)
    for g in (*graphs, *graphs):
        g.replay()
    want = X.experts_block_fp8(xd, idd, wd, *codes)
    for o in outs:
        assert torch.equal(o, want)


@pytest.mark.parametrize("T", [2, 200])
def test_routed_layer_trains_its_router(T):
    """Router, routing and experts together, as a layer: output and gradients by the formulas."""
    E, k, K, I = 6, 2, 128, 144
    x, w13, w2, _, _, dy = _case(T, E, k, K, I, torch.bfloat16, seed=11)
    gate = torch.randn(E, K, generator=torch.Generator().manual_seed(2)) * 0.2
    layer = X.RoutedExperts(X.ExpertsBlockFp8.from_weights(w13.to(DEV), w2.to(DEV)), k, gate, balance=True, score="sigmoid",
                            n_groups=3, top_groups=2, scale=1.5)
    layer.balance.copy_(torch.linspace(-0.1, 0.1, E))
    xd = x.to(DEV).requires_grad_(True)
    y = layer(xd)
    y.backward(dy.to(DEV))
    logits = torch.nn.functional.linear(x.to(DEV).float(), gate.to(DEV)).cpu()     # as the layer formed them
    rw, ri, P = R.route(logits, k, layer.balance.cpu(), "sigmoid", 3, 2, True, 1.5)
    e = layer.experts
    W1 = [R.codes_value(e.CB13[i, 0], e.S13[i, 0]) for i in range(E)]
    W3 = [R.codes_value(e.CB13[i, 1], e.S13[i, 1]) for i in range(E)]
    W2 = [R.codes_value(e.CB2[i], e.S2[i]) for i in range(E)]
    ry, rdx, rdw = R.experts(x, ri, rw.float(), W1, W3, W2, dy)
    by, bx, bw = _bounds(x, ri, rw.float(), W1, W3, W2, dy, ry, rdx, rdw, torch.bfloat16)
    R.check(y, ry, by, "y")
    dl = R.route_grad(P, ri, rdw, "sigmoid", True, 1.5)
    dgate = dl.T @ x.double()
    # an error bw of dw reaches the logits by at most 2 * 1.5 / 4 of the row's largest
    el = 0.75 * bw.sum(1, keepdim=True) + 2.0 ** -22 * dl.abs().amax(1, keepdim=True)
    bound = el.T @ x.double().abs() + (T + 2) * 2.0 ** -23 * (dl.abs().T @ x.double().abs())
    R.check(layer.gate.grad, dgate, bound.expand_as(dgate), "dgate")
    total = rdx + dl @ gate.double()
    extra = el * gate.double().abs().sum(0)[None] + 8 * 2.0 ** -23 * (dl.abs() @ gate.double().abs())
    two = R.half_step(torch.bfloat16) * (rdx.abs() + (dl @ gate.double()).abs() + total.abs()) * 1.02
    R.check(xd.grad, total, bx + extra + two + 1e-30, "dx")


def test_from_linears_and_state_dict(tmp_path):
    torch.manual_seed(1)
    mk = lambda o, i: torch.nn.Linear(i, o, bias=False).to(DEV, torch.bfloat16)  # noqa: E731
    gates, ups, downs = [mk(144, 128) for _ in range(3)], [mk(144, 128) for _ in range(3)], [mk(128, 144) for _ in range(3)]
    m = X.ExpertsBlockFp8.from_linears(gates, ups, downs)
    rq, rs = R.quant_tiles(ups[2].weight.detach().cpu())
    assert torch.equal(m.CB13[2, 1].cpu().view(torch.float8_e4m3fn).double(), rq) and torch.equal(m.S13[2, 1].cpu().double(), rs)
    x, _, _, idx, w, _ = _case(10, 3, 2, 128, 144, torch.bfloat16)
    y = m(x.to(DEV).view(2, 5, 128), idx.to(DEV).view(2, 5, 2), w.to(DEV).view(2, 5, 2))
    torch.save(m.state_dict(), tmp_path / "e.pt")
    n = X.ExpertsBlockFp8(3, 128, 144, device=DEV)
    n.load_state_dict(torch.load(tmp_path / "e.pt"))
    assert torch.equal(n(x.to(DEV), idx.to(DEV), w.to(DEV)).view(2, 5, 128), y)
    assert m(x[:0].to(DEV), idx[:0].to(DEV), w[:0].to(DEV)).shape == (0, 128)


@pytest.mark.parametrize("T", [6, 700])
def test_calls_beside_one_another_on_two_streams(T):
    """Each call has its own counters and partial tiles: interleaved calls change nothing."""
    cases = [_case(T, 4, 2, 512, 272, torch.bfloat16, seed=s) for s in (1, 2)]
    codes, *_ = _codes(cases[0][1], cases[0][2])
    args = [(c[0].to(DEV), c[3].to(DEV), c[4].to(DEV)) for c in cases]
    want = [X.experts_block_fp8(x, i, w, *codes) for x, i, w in args]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(X.experts_block_fp8(*args[k], *codes))
    torch.cuda.synchronize()
    for k in range(2):
        for y in got[k]:
            assert torch.equal(y, want[k])


def test_backward_captured_while_an_eager_graph_lives():
    x, w13, w2, idx, w, dy = _case(50, 4, 2, 256, 144, torch.bfloat16)
    codes, *_ = _codes(w13, w2)
    leaves = [x.to(DEV).requires_grad_(True), w.to(DEV).requires_grad_(True)]
    idd, dyd = idx.to(DEV), dy.to(DEV)
    eager = X.experts_block_fp8(leaves[0], idd, leaves[1], *codes)
    own = [v.detach().clone().requires_grad_(True) for v in leaves]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(X.experts_block_fp8(own[0], idd, own[1], *codes), own, dyd)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        grads = torch.autograd.grad(X.experts_block_fp8(own[0], idd, own[1], *codes), own, dyd)
    g.replay()
    want = torch.autograd.grad(eager, leaves, dyd)
    torch.cuda.synchronize()
    for a, c in zip(grads, want):
        assert torch.equal(a, c)


def test_gradients_against_differences():
    """dw by central differences of the layer itself (it is linear in the weights); dx along a
    direction that the codes hold: see the linear layer's test for the products."""
    x, w13, w2, idx, w, dy = _case(12, 3, 2, 128, 128, torch.bfloat16, none=0.0)
    codes, W1, W3, W2 = _codes(w13, w2)
    wd = w.to(DEV).requires_grad_(True)
    X.experts_block_fp8(x.to(DEV), idx.to(DEV), wd, *codes).backward(dy.to(DEV))
    for t, j in ((0, 0), (5, 1), (11, 0)):
        up, down = w.clone(), w.clone()
        up[t, j] += 0.5
        down[t, j] -= 0.5
        # the formula's dw uses q(dy); the differences take the same
        fu, fd = (R.experts(x, idx, v, W1, W3, W2) for v in (up, down))
        slope = float(((fu - fd) * R.rows_value(dy)).sum())
        # dw stands for h, unquantised; the layer's output for q(h): 2^-4 of each of its terms
        e = int(idx[t, j])
        xq = R.rows_value(x)[t]
        g, u = W1[e] @ xq, W3[e] @ xq
        h = g * torch.sigmoid(g) * u
        terms = (R.rows_value(dy)[t] @ W2[e]) * h
        assert abs(float(wd.grad[t, j]) - slope) <= 2.0 ** -4 * float(terms.abs().sum()) + 1e-6


def test_many_rows_of_one_expert_among_many_experts():
    """Few rows an expert on average, so the weights stream; one expert has several row tiles."""
    x, w13, w2, idx, w, dy = _case(70, 24, 1, 144, 272, torch.bfloat16, none=0.0)
    idx[:, 0] = 17
    idx[::9, 0] = 23
    codes, W1, W3, W2 = _codes(w13, w2)
    y, dx, dw = R.experts(x, idx, w, W1, W3, W2, dy)
    by, bx, bw = _bounds(x, idx, w, W1, W3, W2, dy, y, dx, dw, torch.bfloat16)
    xd, wd = x.to(DEV).requires_grad_(True), w.to(DEV).requires_grad_(True)
    out = X.experts_block_fp8(xd, idx.to(DEV), wd, *codes)
    out.backward(dy.to(DEV))
    R.check(out, y, by)
    R.check(xd.grad, dx, bx)
    R.check(wd.grad, dw, bw)
