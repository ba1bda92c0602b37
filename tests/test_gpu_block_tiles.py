"""The wide product where every CTA pair runs several tiles in a row, in each of its forms, many
experts, and experts' codes and rows past 2^31, on the GPU against 64-bit values.

Bounds.  The fp32 arithmetic's are those of block_ref.py.  Between an expert's two products h is
coded again: a value that fp32 leaves within +-e of h may take any code from that of h - e to that
of h + e, and its block's scale moves with the block's maximum; `moved` is the most that the coded
value can differ by, and goes through the second product as an error of its input.  The same for
the gradients dg and du.  Every row of every output is checked.
"""
import pytest
import torch

from bit_matmul_decomposition_b200 import abi
from bit_matmul_decomposition_b200 import block as B
from bit_matmul_decomposition_b200 import experts as X
from tests import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAIRS = 74                                                 # CTA pairs of the device


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


def _values(codes, scales):
    """codes_value, on the GPU."""
    N, K = codes.shape
    s = scales.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return codes.view(torch.float8_e4m3fn).double() * s


def _rows(v):
    return R.rows_value(v.cpu()).to(DEV)


def _moved(v, ev):
    """How far the coded value of v [rows, C] can move when each element moves by up to ev."""
    v, ev = v.cpu(), ev.cpu()
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], 128):
        t, e = v[:, c:c + 128], ev[:, c:c + 128]
        a = t.abs().amax(1, keepdim=True).clamp_min(R.FLOOR)
        rel = e.amax(1, keepdim=True) / a
        assert (rel < 0.25).all()
        rel = rel / (1 - rel) + 2.0 ** -21
        u = t * 448 / a
        du = (e * 448 / a) * (1 + rel) + u.abs() * rel
        q, lo, hi = R.e4m3(u), R.e4m3(u - du), R.e4m3(u + du)
        out[:, c:c + 128] = (torch.maximum(hi - q, q - lo) * (1 + rel) + q.abs() * rel) * a / 448
    return out.to(DEV)


def _experts(x, idx, w, codes, dy, dtype):
    """y, dx, dw and their bounds, expert by expert in 64 bits on the GPU."""
    CB13, S13, CB2, S2 = codes
    (T, K), k, I = x.shape, idx.shape[1], CB13.shape[2]
    fk, fi = (-(-K // 128) + 40) * 2.0 ** -23, (-(-I // 128) + 40) * 2.0 ** -23
    fc = (k + 1) * 2.0 ** -24                              # the sum over a token's choices
    xq, dyq, w, idx = _rows(x), _rows(dy), w.double().to(DEV), idx.to(DEV)
    y, by, dx, bx = (torch.zeros((T, K), dtype=torch.float64, device=DEV) for _ in range(4))
    dw, bw = (torch.zeros((T, k), dtype=torch.float64, device=DEV) for _ in range(2))
    for e in idx.unique().tolist():
        if e < 0:
            continue
        t, j = torch.nonzero(idx == e, as_tuple=True)
        W1, W3, W2 = _values(CB13[e, 0], S13[e, 0]), _values(CB13[e, 1], S13[e, 1]), _values(CB2[e], S2[e])
        xe, wt = xq[t], w[t, j][:, None]
        g, u = xe @ W1.T, xe @ W3.T
        eg, eu = fk * (xe.abs() @ W1.abs().T), fk * (xe.abs() @ W3.abs().T)
        s = torch.sigmoid(g)
        h = g * s * u
        # |silu'| <= 1.1; the activation is a few steps of fp32; 1.01 for products of two errors
        eh = 1.01 * (1.1 * eg * u.abs() + (g * s).abs() * eu) + 2.0 ** -20 * h.abs()
        hq, mh = _rows(h), _moved(h, eh)
        v = hq @ W2.T
        bv = fi * ((hq.abs() + mh) @ W2.abs().T) + mh @ W2.abs().T
        y.index_add_(0, t, wt * v)
        by.index_add_(0, t, wt.abs() * (bv + fc * v.abs()))
        d = dyq[t]
        dh = d @ W2
        ed = fk * (d.abs() @ W2.abs())
        dw[t, j] = (dh * h).sum(1)
        bw[t, j] = 1.01 * (ed * h.abs() + dh.abs() * eh).sum(1) + (I + 40) * 2.0 ** -24 * (dh * h).abs().sum(1)
        ds = s * (1 + g * (1 - s))                         # its derivative is at most 0.5
        dg, du = wt * dh * u * ds, wt * dh * g * s
        edg = 1.01 * wt.abs() * (ed * (u * ds).abs() + dh.abs() * (eu * 1.1 + u.abs() * 0.5 * eg)) + 2.0 ** -20 * (wt * dh * u).abs()
        edu = 1.01 * wt.abs() * (ed * (g * s).abs() + dh.abs() * 1.1 * eg) + 2.0 ** -20 * du.abs()
        for val, ev, W in ((dg, edg, W1), (du, edu, W3)):
            q, m = _rows(val), _moved(val, ev)
            v = q @ W
            dx.index_add_(0, t, v)
            bx.index_add_(0, t, 2 * fi * ((q.abs() + m) @ W.abs()) + m @ W.abs() + fc * v.abs())
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    hs = R.half_step(dtype) * 1.01
    return [v.cpu() for v in (y, by + hs * (y.abs() + by) + tiny, dx, bx + hs * (dx.abs() + bx) + tiny, dw,
                              bw + 2.0 ** -24 * dw.abs() + 1e-30)]


def _check_experts(x, idx, w, codes, dy):
    y, by, dx, bx, dw, bw = _experts(x, idx, w, codes, dy, x.dtype)
    xd, wd = x.to(DEV).requires_grad_(True), w.to(DEV).requires_grad_(True)
    with torch.no_grad():
        alone = X.experts_block_fp8(xd, idx.to(DEV), wd, *codes)
    out = X.experts_block_fp8(xd, idx.to(DEV), wd, *codes)
    out.backward(dy.to(DEV))
    R.check(alone, y, by, "y without gradients")
    R.check(out, y, by, "y")
    R.check(xd.grad, dx, bx, "dx")
    R.check(wd.grad, dw, bw, "dw")


def _case(T, E, k, K, I, dtype, seed, skew=1.0, none=0.05):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g).to(dtype)
    x[:, ::37] *= 8
    w13 = (torch.randn(E, 2, I, K, generator=g) * 0.06).to(dtype)
    w2 = (torch.randn(E, K, I, generator=g) * 0.06).to(dtype)
    pop = torch.randn(T, E, generator=g) + skew * torch.randn(E, generator=g)
    idx = pop.topk(k, dim=1).indices.to(torch.int32)
    idx[torch.rand(T, k, generator=g) < none] = -1
    w = torch.rand(T, k, generator=g)
    dy = (torch.randn(T, K, generator=g) * 0.1).to(dtype)
    return x, idx, w, (*B.quantize_weight_blocks(w13.to(DEV)), *B.quantize_weight_blocks(w2.to(DEV))), dy


# ------------------------------------------------------------------ many tiles a CTA pair
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_experts_of_many_tiles(dtype):
    T, E, k, K, I = 1700, 8, 2, 2320, 2320
    x, idx, w, codes, dy = _case(T, E, k, K, I, dtype, 3)
    rows = torch.bincount(idx.flatten().long() + 1, minlength=E + 1)[1:]
    m = int((-(-rows // 256)).sum())
    assert rows.max() > 2 * rows.min()
    # the gated product, W2's, dy W2, dg W1 + du W3
    assert min(m * -(-I // 128), m * -(-K // 256), m * -(-I // 256)) > 2 * PAIRS
    _check_experts(x, idx, w, codes, dy)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,K,N", [(300, 2576, 4301), (130, 2560, 4352)])
def test_training_step_of_many_tiles(T, K, N, dtype):
    assert -(-N // 256) * -(-K // 256) > 2 * PAIRS
    g = torch.Generator().manual_seed(T)
    x, dy = torch.randn(T, K, generator=g).to(dtype), (torch.randn(T, N, generator=g) * 1e-2).to(dtype)
    w = (torch.randn(N, K, generator=g) * 0.05).to(dtype)
    leaves = [v.to(DEV).requires_grad_(True) for v in (x, w)]
    B.linear_block_fp8_train(*leaves).backward(dy.to(DEV))
    gt, xt = R.tiles_value(dy), R.tiles_value(x)
    ref = gt.T @ xt
    R.check(leaves[1].grad, ref, R.product_bound(gt.T, xt.T, dtype, ref, T), "dw")
    gv, wv = R.rows_value(dy), R.tiles_value(w)
    ref = gv @ wv
    R.check(leaves[0].grad, ref, R.product_bound(gv, wv.T, dtype, ref, N), "dx")


@pytest.mark.parametrize("N", [5000, 5001])                # outputs that leave by TMA, and row by row
def test_layer_of_many_tiles(N):
    T, K = 2100, 400
    assert -(-T // 256) * -(-N // 256) > 2 * PAIRS
    g = torch.Generator().manual_seed(N)
    x, w = torch.randn(T, K, generator=g).to(torch.bfloat16), (torch.randn(N, K, generator=g) * 0.05).to(torch.bfloat16)
    b = torch.randn(N, generator=g).to(torch.bfloat16)
    codes, scales = B.quantize_weight_blocks(w.to(DEV))
    xv, wv = R.rows_value(x), R.codes_value(codes, scales)
    ref = xv @ wv.T + b.double()
    R.check(B.linear_block_fp8(x.to(DEV), codes, scales, b.to(DEV)), ref,
            R.product_bound(xv, wv, torch.bfloat16, ref, K) + 2.0 ** -23 * b.double().abs())
    dy = (torch.randn(T, N, generator=g) * 1e-2).to(torch.bfloat16)
    xd = x.to(DEV).requires_grad_(True)
    B.linear_block_fp8(xd, codes, scales, b.to(DEV)).backward(dy.to(DEV))
    gv = R.rows_value(dy)
    ref = gv @ wv
    R.check(xd.grad, ref, R.product_bound(gv, wv.T, torch.bfloat16, ref, N), "dx")


# ------------------------------------------------------------------ many experts
@pytest.mark.parametrize("T,E,k", [(130, 256, 6), (700, 256, 8), (60, 512, 8), (1100, 300, 4)])
def test_many_experts(T, E, k):
    """Fewer rows an expert than the streaming product's limit, and more."""
    _check_experts(*_case(T, E, k, 144, 48, torch.bfloat16, E + T))


# ------------------------------------------------------------------ past 32 bits
@pytest.mark.parametrize("T", [40, 1200])                  # streaming, and in tiles
def test_experts_of_more_than_2_31_codes(T):
    E, K, I = 130, 4096, 4096                              # CB13 4.4e9 codes, CB2 2.2e9
    g = torch.Generator(device=DEV).manual_seed(1)

    def codes(*shape):
        c = torch.empty(shape, dtype=torch.uint8, device=DEV)
        for e in range(E):
            c[e] = torch.randint(0, 256, shape[1:], generator=g, device=DEV, dtype=torch.uint8) & 0xBF
        return c
    all_codes = (codes(E, 2, I, K), 0.02 * torch.rand((E, 2, 32, 32), generator=g, device=DEV),
                 codes(E, K, I), 0.02 * torch.rand((E, 32, 32), generator=g, device=DEV))
    c = torch.Generator().manual_seed(2)
    x, dy = torch.randn(T, K, generator=c).to(torch.bfloat16), torch.randn(T, K, generator=c).to(torch.bfloat16)
    idx = torch.tensor([0, 60, E - 2, E - 1], dtype=torch.int32)[torch.randint(0, 4, (T, 1), generator=c)]
    _check_experts(x, idx, torch.rand(T, 1, generator=c), all_codes, dy)


def test_experts_rows_of_more_than_2_31_elements():
    """g and u, and the codes of dg and du, past 2^31; the last tokens repeat the first."""
    T, E, K, I = 140000, 2, 16, 8192
    _, _, _, codes, _ = _case(4, E, 1, K, I, torch.bfloat16, 9)
    g = torch.Generator(device=DEV).manual_seed(4)
    x, dy = (torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    idx = torch.randint(0, E, (T, 1), generator=g, device=DEV, dtype=torch.int32)
    w = torch.rand(T, 1, generator=g, device=DEV)
    for v in (x, dy, idx, w):
        v[-300:] = v[:300]
    assert T * 2 * I > 1 << 31
    xd, wd = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    out = X.experts_block_fp8(xd, idx, wd, *codes)
    out.backward(dy)
    for v in (out, xd.grad, wd.grad):
        assert torch.isfinite(v).all() and torch.equal(v[-300:], v[:300])
    last = [v[-40:].cpu() for v in (x, idx, w, dy)]
    y, by, dx, bx, dw, bw = _experts(last[0], last[1], last[2], codes, last[3], torch.bfloat16)
    R.check(out[-40:], y, by, "y")
    R.check(xd.grad[-40:], dx, bx, "dx")
    R.check(wd.grad[-40:], dw, bw, "dw")
