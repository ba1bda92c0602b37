"""The block-scaled e4m3 linear layer on the GPU against the 64-bit reference: codes and scales
bit for bit, forward, gradients, and the calls that a user may make of them."""
import pytest
import torch

from bit_matmul_decomposition_b200 import abi
from bit_matmul_decomposition_b200 import block as B
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


def _x(T, K, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g) * torch.exp(0.5 * torch.randn(T, 1, generator=g))
    x[:, :: max(1, K // 3)] *= 30.0
    return x.to(dtype)


def _w(N, K, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(N, K, generator=g) * 0.05).to(dtype)


def _act_codes(x):
    T, K = x.shape
    q = torch.full((T, K), 77, dtype=torch.uint8, device=DEV)
    s = torch.full((-(-K // 128), T), float("nan"), device=DEV)
    abi.i8_block_quantize_act(x, q, s)
    return q.cpu(), s.cpu()


# ------------------------------------------------------------------ codes and scales
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,K", [(1, 16), (1, 4096), (3, 144), (129, 256), (200, 1040)])
def test_activation_codes_bit_for_bit(T, K, dtype):
    x = _x(T, K, dtype)
    x[0, 0] = 0.0
    if T > 2:
        x[2] = 0.0
    q, s = _act_codes(x.to(DEV))
    rq, rs = R.quant_rows(x)
    assert torch.equal(q.view(torch.float8_e4m3fn).double(), rq)
    assert torch.equal(s.T.double(), rs)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,K", [(1, 16), (130, 144), (257, 400), (64, 1024)])
def test_weight_codes_bit_for_bit(N, K, dtype):
    w = _w(N, K, dtype)
    w[0, :16] *= 100
    q, s = B.quantize_weight_blocks(w.to(DEV))
    rq, rs = R.quant_tiles(w)
    assert torch.equal(q.cpu().view(torch.float8_e4m3fn).double(), rq)
    assert torch.equal(s.cpu().double(), rs)


def test_weight_codes_of_a_stack():
    w = torch.stack([torch.stack([_w(40, 144, torch.bfloat16, s), _w(40, 144, torch.bfloat16, s + 9)]) for s in range(3)])
    q, s = B.quantize_weight_blocks(w.to(DEV))
    assert q.shape == (3, 2, 40, 144) and s.shape == (3, 2, 1, 2)
    for i in range(3):
        for j in range(2):
            rq, rs = R.quant_tiles(w[i, j])
            assert torch.equal(q[i, j].cpu().view(torch.float8_e4m3fn).double(), rq)
            assert torch.equal(s[i, j].cpu().double(), rs)


def test_codes_at_the_ends_of_the_range():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    x[0, 5] = 3e38                        # the largest a
    x[1, 7] = 1e-38                       # below the floor: codes 0
    x[2, :3] = torch.tensor([2.0 ** -100, 2.0 ** -101, -(2.0 ** -100)], dtype=torch.bfloat16)
    x[3] = -448.0
    q, s = _act_codes(x.to(DEV))
    rq, rs = R.quant_rows(x)
    assert torch.equal(q.view(torch.float8_e4m3fn).double(), rq) and torch.equal(s.T.double(), rs)
    h = torch.zeros(2, 16, dtype=torch.float16)
    h[0, 0], h[0, 1] = 6e-8, 65504.0
    h[1, 3] = 6e-8                        # the smallest fp16 value alone in its block
    q, s = _act_codes(h.to(DEV))
    rq, rs = R.quant_rows(h)
    assert torch.equal(q.view(torch.float8_e4m3fn).double(), rq) and torch.equal(s.T.double(), rs)
    assert rq[1, 3] == 448.0


# ------------------------------------------------------------------ forward
def _forward_case(T, K, N, dtype, bias, seed=0):
    x, w = _x(T, K, dtype, seed), _w(N, K, dtype, seed + 1)
    b = _x(1, N, dtype, seed + 2)[0] if bias else None
    codes, scales = B.quantize_weight_blocks(w.to(DEV))
    xv, wv = R.rows_value(x), R.codes_value(codes, scales)
    ref = xv @ wv.T
    bound = R.product_bound(xv, wv, dtype, ref + (b.double() if bias else 0.0), K)
    if bias:
        ref = ref + b.double()
        bound = bound + 2.0 ** -23 * b.double().abs()
    return x.to(DEV), codes, scales, None if b is None else b.to(DEV), ref, bound


SHAPES = [(1, 16, 1), (1, 64, 64), (2, 128, 130), (13, 4096, 700), (16, 144, 129), (17, 272, 40), (32, 1040, 333),
          (33, 256, 256), (64, 512, 1000), (65, 4112, 129), (128, 384, 257), (129, 128, 128), (256, 256, 256),
          (300, 1040, 605), (513, 2064, 777), (1, 16384, 3), (700, 16, 8)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_forward(T, K, N, dtype):
    bias = (T + N) % 2 == 1
    x, codes, scales, b, ref, bound = _forward_case(T, K, N, dtype, bias)
    R.check(B.linear_block_fp8(x, codes, scales, b), ref, bound)


@pytest.mark.parametrize("T", [1, 20, 128, 200])
def test_forward_writes_its_rows_alone_and_the_same_every_time(T):
    K, N = 1040, 520
    x, codes, scales, _, ref, bound = _forward_case(T, K, N, torch.bfloat16, False)
    ws = torch.full((abi.i8_block_linear_workspace_size(T, N, K),), 255, dtype=torch.uint8, device=DEV)
    big = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    first = None
    for _ in range(3):                    # the workspace starts with whatever the last call left
        abi.i8_block_linear_forward(x, codes, scales, None, big[1:T + 1], ws)
        got = big.clone()
        assert (got[0] == 7).all() and (got[T + 1] == 7).all()
        first = got if first is None else first
        assert torch.equal(first, got)
    R.check(first[1:T + 1], ref, bound)


@pytest.mark.parametrize("T", [5, 300])
def test_not_finite_values_stay_in_their_row(T):
    K, N = 400, 140
    x, codes, scales, _, ref, bound = _forward_case(T, K, N, torch.float16, False)
    x[1, 3], x[2, 399], x[4, 200] = float("inf"), float("nan"), float("-inf")
    y = B.linear_block_fp8(x, codes, scales)
    bad = [1, 2, 4]
    assert torch.isnan(y[bad]).all()
    keep = [t for t in range(T) if t not in bad]
    R.check(y[keep], ref[keep], bound[keep])


def test_a_nan_code_of_the_weight_stays_in_its_column():
    x, codes, scales, _, ref, bound = _forward_case(40, 256, 200, torch.bfloat16, False)
    codes[150, 17] = 0x7F
    y = B.linear_block_fp8(x, codes, scales)
    assert torch.isnan(y[:, 150]).all()
    keep = [n for n in range(200) if n != 150]
    R.check(y[:, keep], ref[:, keep], bound[:, keep])


def test_stored_scales_of_any_size_and_sign_of_code():
    """Scales as a checkpoint may hold them: not powers of two, unlike from tile to tile."""
    T, K, N = 70, 384, 300
    g = torch.Generator().manual_seed(5)
    codes = torch.randint(0, 256, (N, K), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0
    scales = torch.exp(2 * torch.randn(3, 3, generator=g)) * 1e-3
    x = _x(T, K, torch.bfloat16)
    m = B.LinearBlockFp8.from_codes(codes.to(DEV).view(torch.float8_e4m3fn), scales.to(DEV))
    xv, wv = R.rows_value(x), R.codes_value(codes, scales)
    ref = xv @ wv.T
    R.check(m(x.to(DEV)), ref, R.product_bound(xv, wv, torch.bfloat16, ref, K))


def test_strided_offset_and_batched_inputs():
    x, codes, scales, b, ref, bound = _forward_case(24, 256, 100, torch.float16, True)
    wide = torch.zeros(24, 512, dtype=torch.float16, device=DEV)
    wide[:, ::2] = x
    y = B.linear_block_fp8(wide[:, ::2].view(2, 12, 256), codes, scales, b)
    assert y.shape == (2, 12, 100)
    R.check(y.view(24, 100), ref, bound)
    flat = torch.zeros(24 * 256 + 3, dtype=torch.float16, device=DEV)
    flat[3:] = x.flatten()
    R.check(B.linear_block_fp8(flat[3:].view(24, 256), codes, scales, b), ref, bound)
    assert B.linear_block_fp8(x[:0], codes, scales, b).shape == (0, 100)
    assert B.linear_block_fp8(x[0], codes, scales, b).shape == (100,)


def test_another_stream():
    x, codes, scales, b, ref, bound = _forward_case(16, 2048, 512, torch.bfloat16, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ys = []
    with torch.cuda.stream(s):
        for _ in range(4):
            ys.append(B.linear_block_fp8(x, codes, scales, b))
    y0 = B.linear_block_fp8(x, codes, scales, b)          # beside the other stream's calls
    torch.cuda.synchronize()
    for y in (*ys, y0):
        R.check(y, ref, bound)


@pytest.mark.parametrize("T", [3, 150])
def test_captured_and_replayed(T):
    K, N = 1024, 300
    x, codes, scales, b, ref, bound = _forward_case(T, K, N, torch.bfloat16, True)
    x2, _, _, _, ref2, bound2 = _forward_case(T, K, N, torch.bfloat16, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.linear_block_fp8(x, codes, scales, b)
    torch.cuda.current_stream().wait_stream(s)
    graphs, outs = [], []
    xin = x.clone()
    for _ in range(2):                                     # two graphs, each with its workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(B.linear_block_fp8(xin, codes, scales, b))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    for o in outs:
        R.check(o, ref, bound)
    y3 = _x(T, K, torch.bfloat16, seed=44)
    xin.copy_(y3)
    for g in graphs:
        g.replay()
    xv, wv = R.rows_value(y3), R.codes_value(codes, scales)
    r3 = xv @ wv.T + b.cpu().double()
    for o in outs:
        R.check(o, r3, R.product_bound(xv, wv, torch.bfloat16, r3, K) + 2.0 ** -23 * b.cpu().double().abs())


# ------------------------------------------------------------------ gradients
def _step_case(T, K, N, dtype, seed=0):
    x, w = _x(T, K, dtype, seed), _w(N, K, dtype, seed + 1)
    b = _x(1, N, dtype, seed + 2)[0]
    g = torch.Generator().manual_seed(seed + 3)
    dy = (torch.randn(T, N, generator=g) * torch.exp(torch.randn(T, 1, generator=g)) * 1e-2).to(dtype)
    return x, w, b, dy


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,K,N", [(1, 16, 1), (5, 144, 40), (128, 128, 128), (130, 272, 257), (300, 1040, 605), (260, 512, 264)])
def test_training_step(T, K, N, dtype):
    x, w, b, dy = _step_case(T, K, N, dtype)
    leaves = [v.to(DEV).requires_grad_(True) for v in (x, w, b)]
    y = B.linear_block_fp8_train(*leaves)
    y.backward(dy.to(DEV))
    wv, xv = R.tiles_value(w), R.rows_value(x)
    ref = xv @ wv.T + b.double()
    R.check(y, ref, R.product_bound(xv, wv, dtype, ref, K) + 2.0 ** -23 * b.double().abs(), "y")
    gv = R.rows_value(dy)
    ref = gv @ wv
    R.check(leaves[0].grad, ref, R.product_bound(gv, wv.T, dtype, ref, N), "dx")
    gt, xt = R.tiles_value(dy), R.tiles_value(x)
    ref = gt.T @ xt
    R.check(leaves[1].grad, ref, R.product_bound(gt.T, xt.T, dtype, ref, T), "dw")
    ref = dy.double().sum(0)
    R.check(leaves[2].grad, ref, R.half_step(dtype) * ref.abs() * (1 + 2.0 ** -12) + T * 2.0 ** -24 * dy.double().abs().sum(0)
            + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2, "db")


def test_only_the_wanted_gradients_and_frozen_codes():
    T, K, N = 40, 256, 136
    x, w, b, dy = _step_case(T, K, N, torch.bfloat16)
    wv = R.tiles_value(w)
    gv = R.rows_value(dy)
    ref = gv @ wv
    bound = R.product_bound(gv, wv.T, torch.bfloat16, ref, N)
    lin = torch.nn.Linear(K, N).to(DEV, torch.bfloat16)
    with torch.no_grad():
        lin.weight.copy_(w)
        lin.bias.copy_(b)
    frozen = B.LinearBlockFp8.from_linear(lin)
    xd = x.to(DEV).requires_grad_(True)
    frozen(xd).backward(dy.to(DEV))
    R.check(xd.grad, ref, bound)
    train = B.LinearBlockFp8.from_linear(lin, has_16bit_weights=True)
    y = train(x.to(DEV))                                   # x needs no gradient
    y.backward(dy.to(DEV))
    gt, xt = R.tiles_value(dy), R.tiles_value(x)
    r = gt.T @ xt
    R.check(train.weight.grad, r, R.product_bound(gt.T, xt.T, torch.bfloat16, r, T))
    train.weight.requires_grad_(False)
    train.zero_grad()
    train.bias.grad = None
    train(x.to(DEV)).sum().backward()                      # an expanded gradient; bias alone
    assert torch.equal(train.bias.grad, torch.full((N,), float(T), dtype=torch.bfloat16, device=DEV))
    with torch.no_grad():
        assert torch.equal(train(xd), frozen(xd))
    e = torch.zeros((0, K), dtype=torch.bfloat16, device=DEV, requires_grad=True)
    train.weight.requires_grad_(True)
    train(e).sum().backward()
    assert e.grad.shape == (0, K) and (train.weight.grad == 0).all()


def test_gradients_against_differences():
    """On inputs that the codes hold exactly the layer is linear, and a step along one of them
    changes the output by exactly the gradient: every block has its 448 2^j and small integers."""
    T, K, N = 20, 256, 144
    g = torch.Generator().manual_seed(3)
    def exact(*shape):
        v = torch.randint(-15, 16, shape, generator=g).float()
        v[::1, ::128] = 448.0                              # fixes every block's and tile's scale at 1
        return v
    x, w, dy = exact(T, K), exact(N, K), exact(T, N)
    leaves = [v.to(DEV, torch.bfloat16).requires_grad_(True) for v in (x, w)]
    y = B.linear_block_fp8_train(*leaves)
    f0 = (R.rows_value(x) @ R.tiles_value(w).T * dy.double()).sum()
    y.backward(dy.to(DEV, torch.bfloat16))
    for leaf, v, which in ((leaves[0], x, 0), (leaves[1], w, 1)):
        for i, j in ((0, 1), (7, 130), (19, 255)):
            step = v.clone()
            step[i, j] += 1.0 if step[i, j] < 15 else -1.0
            d = float(step[i, j] - v[i, j])
            a, b = (step, w) if which == 0 else (x, step)
            f1 = ((R.rows_value(a) @ R.tiles_value(b).T) * dy.double()).sum()
            slope = float(f1 - f0) / d
            assert abs(float(leaf.grad[i, j]) - slope) <= R.half_step(torch.bfloat16) * abs(slope) * 1.01, (which, i, j)


def test_backward_captured_while_an_eager_graph_lives():
    T, K, N = 40, 256, 136
    x, w, b, dy = _step_case(T, K, N, torch.bfloat16)
    leaves = [v.to(DEV).requires_grad_(True) for v in (x, w, b)]
    dyd = dy.to(DEV)
    eager = B.linear_block_fp8_train(*leaves)              # lives across the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        own = [v.detach().clone().requires_grad_(True) for v in leaves]
        torch.autograd.grad(B.linear_block_fp8_train(*own), own, dyd)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        grads = torch.autograd.grad(B.linear_block_fp8_train(*own), own, dyd)
    g.replay()
    want = torch.autograd.grad(eager, leaves, dyd)
    torch.cuda.synchronize()
    for a, c in zip(grads, want):
        assert torch.equal(a, c)


def test_replace_and_state_dict(tmp_path):
    torch.manual_seed(0)
    m = torch.nn.Sequential()
    m.add_module("up", torch.nn.Linear(128, 200))
    m.add_module("lm_head", torch.nn.Linear(200, 10))
    m = m.to(DEV, torch.bfloat16)
    w = m.up.weight.detach().cpu()
    B.replace_linear_with_block_fp8(m)
    assert isinstance(m.up, B.LinearBlockFp8) and isinstance(m.lm_head, torch.nn.Linear)
    x = _x(9, 128, torch.bfloat16)
    y = m.up(x.to(DEV))
    xv, wv = R.rows_value(x), R.tiles_value(w)
    ref = xv @ wv.T + m.up.bias.cpu().double()
    R.check(y, ref, R.product_bound(xv, wv, torch.bfloat16, ref, 128) + 1e-6)
    torch.save(m.up.state_dict(), tmp_path / "l.pt")
    n = B.LinearBlockFp8(128, 200, device=DEV)
    n.load_state_dict(torch.load(tmp_path / "l.pt"))
    assert torch.equal(n(x.to(DEV)), y)


# ------------------------------------------------------------------ sizes past 32 bits
def test_a_weight_of_more_than_2_31_codes():
    """The last rows of the weight repeat the first: so do the last columns of the output."""
    K, N = 20480, 106000                                  # 2.17e9 codes
    g = torch.Generator(device=DEV).manual_seed(1)
    codes = torch.empty((N, K), dtype=torch.uint8, device=DEV)
    for i in range(0, N, 10600):
        codes[i:i + 10600] = torch.randint(0, 256, (10600, K), generator=g, device=DEV, dtype=torch.uint8) & 0xBF
    tail = N - 256 - (N % 128)                            # whole tiles, so that the scales can repeat too
    codes[tail:tail + 256] = codes[:256]
    scales = torch.rand(((N + 127) // 128, K // 128), generator=g, device=DEV)
    scales[tail // 128:tail // 128 + 2] = scales[:2]
    for T in (2, 40, 130):                                # both forms of the product
        x = _x(T, K, torch.bfloat16).to(DEV)
        y = B.linear_block_fp8(x, codes, scales)
        assert torch.isfinite(y).all() and torch.equal(y[:, tail:tail + 256], y[:, :256])
        del x, y
    xv, wv = R.rows_value(_x(2, K, torch.bfloat16)), R.codes_value(codes[tail:tail + 8], scales[tail // 128:tail // 128 + 1])
    ref = xv @ wv.T
    got = B.linear_block_fp8(_x(2, K, torch.bfloat16).to(DEV), codes, scales)[:, tail:tail + 8]
    R.check(got, ref, R.product_bound(xv, wv, torch.bfloat16, ref, K))


def test_activations_and_gradients_of_more_than_2_31_elements():
    T, K, N = 135000, 16384, 16                           # x: 2.2e9 elements
    w = (torch.randn(N, K) * 0.05).to(torch.bfloat16).to(DEV).requires_grad_(True)
    x = torch.empty((T, K), dtype=torch.bfloat16, device=DEV)
    for i in range(0, T, 13500):
        x[i:i + 13500] = torch.randn(13500, K, device=DEV)
    x[-300:] = x[:300]
    x.requires_grad_(True)
    y = B.linear_block_fp8_train(x, w)
    assert torch.equal(y[-300:], y[:300])
    dy = torch.randn(T, N, device=DEV).to(torch.bfloat16)
    dy[-300:] = dy[:300]
    y.backward(dy)
    assert torch.equal(x.grad[-300:], x.grad[:300])
    gv, wv = R.rows_value(dy[-5:].cpu()), R.tiles_value(w.detach().cpu())
    ref = gv @ wv
    R.check(x.grad[-5:], ref, R.product_bound(gv, wv.T, torch.bfloat16, ref, N))
    assert torch.isfinite(w.grad).all()


# ------------------------------------------------------------------ wide layers, few tokens
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,K,N", [(17, 144, 20737), (32, 1040, 20600), (33, 16, 20501), (64, 400, 20483), (65, 256, 20600)])
def test_wide_layers(T, K, N, dtype):
    """More than 80 tiles of 256 outputs: up to 64 tokens stream the weight."""
    x, codes, scales, b, ref, bound = _forward_case(T, K, N, dtype, N % 2 == 1)
    ws = torch.full((abi.i8_block_linear_workspace_size(T, N, K),), 255, dtype=torch.uint8, device=DEV)
    big = torch.full(((T + 2) * N + 16,), 7.0, dtype=dtype, device=DEV)
    y = big[8:8 + T * N].view(T, N)
    abi.i8_block_linear_forward(x, codes, scales, b, y, ws)
    first = y.clone()
    R.check(first, ref, bound)
    abi.i8_block_linear_forward(x, codes, scales, b, y, ws)
    assert torch.equal(first, y) and (big[:8] == 7).all() and (big[8 + T * N:] == 7).all()
    x[T - 2, K - 1] = float("nan")
    z = B.linear_block_fp8(x, codes, scales, b)
    assert torch.isnan(z[T - 2]).all()
    keep = [t for t in range(T) if t != T - 2]
    assert torch.equal(z[keep], first[keep])
