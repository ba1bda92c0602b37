"""Plain 64-bit reference of the block-scaled operators, for the tests: numpy-style torch code
on the CPU, written from the formulas in include/i8linear.h, sharing nothing with the package.

Error bound of a product's element, besides the half step of its 16-bit rounding: with A the sum
of the magnitudes of its terms, every addition on the way is off by at most 2^-23 A (a step of
fp32, truncation allowed).  A block of 128 takes four MMAs of 32 terms: at most 32 + 4 of them;
its scaling two roundings, the sum over the blocks one each, the bias one: (blocks + 40) 2^-23 A.
"""
import math

import torch

FLOOR = 2.0 ** -100


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def e4m3(v):
    """e4m3 value nearest to v, ties to even: 4 significant bits, steps of 2^-9 below 2^-6."""
    _, e = torch.frexp(v)
    step = torch.pow(2.0, (e - 4).clamp_min(-9).double())
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _scale_pair(a):
    a = a.clamp_min(FLOOR)
    up = (448.0 / a).float().double()
    down = (a * torch.tensor(1.0 / 448.0, dtype=torch.float32).double()).float().double()
    return up, down


def quant_rows(v):
    """(values of the codes, scales [.., blocks]) of v [R, C] in row blocks of 128."""
    v = v.double()
    R, C = v.shape
    q, s = torch.zeros_like(v), torch.zeros((R, -(-C // 128)), dtype=torch.float64)
    for b in range(s.shape[1]):
        t = v[:, b * 128:(b + 1) * 128]
        up, down = _scale_pair(t.abs().amax(dim=1))
        q[:, b * 128:(b + 1) * 128] = e4m3((t * up[:, None]).float().double())
        s[:, b] = down
    return q, s


def quant_tiles(v):
    v = v.double()
    R, C = v.shape
    q, s = torch.zeros_like(v), torch.zeros((-(-R // 128), -(-C // 128)), dtype=torch.float64)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            t = v[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]
            up, down = _scale_pair(t.abs().max())
            q[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128] = e4m3((t * up).float().double())
            s[i, j] = down
    return q, s


def spread(s, rows, cols, by_row=False):
    """Scales [.., blocks] as one number per element of a [rows, cols] matrix."""
    s = s.repeat_interleave(128, dim=1)[:, :cols]
    return s if by_row else s.repeat_interleave(128, dim=0)[:rows]


def rows_value(v):
    q, s = quant_rows(v)
    return q * spread(s, *v.shape, by_row=True)


def tiles_value(v):
    q, s = quant_tiles(v)
    return q * spread(s, *v.shape)


def codes_value(codes, scales):
    N, K = codes.shape
    return codes.cpu().view(torch.float8_e4m3fn).double() * spread(scales.cpu().double(), N, K)


def product_bound(a, b, dtype, ref, terms):
    """Largest error allowed for each element of a b^T (a, b in 64 bits)."""
    A = a.abs() @ b.abs().T
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    return half_step(dtype) * ref.abs() * (1 + 2.0 ** -12) + (-(-terms // 128) + 40) * 2.0 ** -23 * A + tiny


def check(got, ref, bound, what=""):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), "%s: non-finite output" % what
    err = (got - ref).abs()
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert (err <= bound).all(), "%s: worst err/allowed = %.3f" % (what, worst)
    return worst


# ------------------------------------------------------------------ routing, token by token
def route(logits, k, balance, score, n_groups, top_groups, renormalize, scale):
    """(weights, idx, scores) by Python floats; logits a [T, E] CPU tensor without NaN."""
    T, E = logits.shape
    W, I, P = [], [], []
    for t in range(T):
        x = [float(v) for v in logits[t].double()]
        live = [v > -math.inf for v in x]
        if score == "softmax":
            m = max(x)
            z = [math.exp(v - m) if ok else 0.0 for v, ok in zip(x, live)]
            s = math.fsum(z)
            p = [v / s if s else 0.0 for v in z]
        else:
            p = [(1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0) if ok else 0.0 for v, ok in zip(x, live)]
        key = {e: p[e] + (float(balance[e]) if balance is not None else 0.0) for e in range(E) if live[e]}
        size = E // n_groups
        if n_groups > 1:
            totals = []
            for g in range(n_groups):
                best = sorted((key[e] for e in range(g * size, (g + 1) * size) if e in key), reverse=True)
                best = best[:2 if balance is not None else 1]
                totals.append(sum(best) if best else -math.inf)
            kept = sorted(range(n_groups), key=lambda g: (-totals[g], g))[:top_groups]
            key = {e: v for e, v in key.items() if e // size in kept}
        order = sorted(key, key=lambda e: (-key[e], e))[:k]
        S = math.fsum(p[e] for e in order)
        w = [(p[e] / S if S > 0 else 0.0) * scale if renormalize else p[e] * scale for e in order]
        W.append(w + [0.0] * (k - len(w)))
        I.append(order + [-1] * (k - len(order)))
        P.append(p)
    return (torch.tensor(W, dtype=torch.float64), torch.tensor(I, dtype=torch.int32),
            torch.tensor(P, dtype=torch.float64))


def route_grad(P, idx, dw, score, renormalize, scale):
    """Gradient of the logits by the formulas, [T, E]."""
    T, E = P.shape
    out = torch.zeros_like(P)
    for t in range(T):
        sel = [(j, int(e)) for j, e in enumerate(idx[t]) if e >= 0]
        g = {j: float(dw[t, j]) * scale for j, _ in sel}
        S = sum(float(P[t, e]) for _, e in sel)
        gs = sum(g[j] * float(P[t, e]) for j, e in sel)
        ds = torch.zeros(E, dtype=torch.float64)
        for j, e in sel:
            if renormalize:
                ds[e] += (g[j] - gs / S) / S if S > 0 else 0.0
            else:
                ds[e] += g[j]
        p = P[t]
        out[t] = p * (ds - (ds * p).sum()) if score == "softmax" else ds * p * (1 - p)
    return out


# ------------------------------------------------------------------ experts
def experts(x, idx, w, W1, W3, W2, dy=None):
    """y, and with dy also dx and dw; W1, W3 [E][I, K] and W2 [E][K, I] in 64 bits."""
    T, K = x.shape
    xq = rows_value(x)
    y, dx = torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    dw = torch.zeros(w.shape, dtype=torch.float64)
    dyq = rows_value(dy) if dy is not None else None
    for e in range(len(W1)):
        for t, j in torch.nonzero(idx == e).tolist():
            g, u = W1[e] @ xq[t], W3[e] @ xq[t]
            sg = torch.sigmoid(g)
            h = g * sg * u
            wt = float(w[t, j])
            y[t] += wt * (W2[e] @ rows_value(h[None])[0])
            if dy is not None:
                dh = dyq[t] @ W2[e]
                dw[t, j] = (dh * h).sum()
                dh = dh * wt
                dg, du = dh * u * sg * (1 + g * (1 - sg)), dh * g * sg
                dx[t] += rows_value(dg[None])[0] @ W1[e] + rows_value(du[None])[0] @ W3[e]
    return (y, dx, dw) if dy is not None else y
