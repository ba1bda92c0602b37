"""Block-scaled 8-bit floating-point operators: their cases, plain forms and 64-bit values.

Three operators, each forward and with its gradients:

  linear    y = x W^T + b with e4m3 codes and one scale for each block: x in blocks of 128
            features per token, W in tiles of 128 x 128 (kinds "linear" and "linear_step")
  route     scores of the experts, balance bias, groups, top-k, weights ("route", "route_step")
  experts   y[t] = sum_j w[t,j] * expert idx[t,j] of x[t], each expert a gated
            feed-forward whose three products are block-scaled ("experts", "experts_step")

A "_step" kind is one training pass: the forward, then the gradients for a given gradient of
the output.  Quantisation passes gradients straight through.

A block's codes are e4m3(fl32(v * fl32(448 / a))) with a = max(largest |v|, 2^-100), and its
scale is fl32(a * fl32(1 / 448)).
"""
import torch

own = False

BLOCK = 128
FLOOR = 2.0 ** -100
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token through a 4096 -> 16384 feed-forward layer: weights are all the traffic
        dict(name="linear_t1", kind="linear", T=1, K=4096, N=16384, dtype="fp16", bias=True),
        # a decode batch on the widest layer that the benchmark has
        dict(name="linear_t13_wide", kind="linear", T=13, K=14336, N=57344, dtype="bf16", bias=True),
        # a short prompt on odd sizes: a partial block of features, an odd number of outputs
        dict(name="linear_t333_odd", kind="linear", T=333, K=4112, N=6007, dtype="fp16", bias=True),
        # a long prompt on the benchmark's headline layer
        dict(name="linear_t2048_large", kind="linear", T=2048, K=12288, N=49152, dtype="bf16", bias=False),
        # training steps: a full batch, and a small ragged one
        dict(name="linear_step_t2048", kind="linear_step", T=2048, K=4096, N=16384, dtype="bf16", bias=True),
        dict(name="linear_step_t300_odd", kind="linear_step", T=300, K=1040, N=605, dtype="fp16", bias=True),
        # routing of a single token (sigmoid scores, balance bias, 4 of 8 groups)
        dict(name="route_t1", kind="route", T=1, E=256, k=8, score="sigmoid", balance=True, groups=8, top_groups=4,
             renorm=True, scale=2.5, dtype="fp32", masked=False),
        # routing of a long prompt, some experts and some padding tokens masked
        dict(name="route_t16384", kind="route", T=16384, E=128, k=8, score="softmax", balance=False, groups=1,
             top_groups=1, renorm=True, scale=1.0, dtype="fp32", masked=True),
        # the router in a training step
        dict(name="route_step_t8192", kind="route_step", T=8192, E=256, k=8, score="sigmoid", balance=True, groups=8,
             top_groups=4, renorm=True, scale=2.5, dtype="bf16", masked=False),
        # one token through its 8 experts: the weights of 8 experts are the traffic
        dict(name="experts_t1", kind="experts", T=1, E=64, k=8, K=4096, I=1024, dtype="bf16", padded=False),
        # a prompt with skewed popularity of the experts and a hidden size that is not whole blocks
        dict(name="experts_t2048", kind="experts", T=2048, E=64, k=6, K=2048, I=1424, dtype="bf16", padded=True),
        # frozen experts inside a model that trains: gradients of the input and of the weights of the routing
        dict(name="experts_step_t1024", kind="experts_step", T=1024, E=32, k=4, K=2048, I=1024, dtype="bf16",
             padded=False),
    ]


def _spread(rng, low, high, unit=1):
    """A whole number of `unit`s between low and high, even over its logarithm."""
    v = low * (high / low) ** rng.random()
    return max(low, min(high, int(round(v / unit)) * unit))


def draw(rng):
    kind = rng.choice(["linear", "linear", "linear_step", "route", "route_step", "experts", "experts_step"])
    half = rng.choice(["bf16", "bf16", "fp16"])
    if kind == "linear":
        K, N = _spread(rng, 64, 14336, 16), _spread(rng, 33, 57344)
        most = int(1.2e12 // (K * N))
        return dict(kind=kind, T=_spread(rng, 1, max(1, min(4096, most))), K=K, N=N, dtype=half, bias=rng.random() < 0.7)
    if kind == "linear_step":
        K, N = _spread(rng, 64, 8192, 16), _spread(rng, 33, 16384)
        most = int(1.3e11 // (K * N))
        return dict(kind=kind, T=_spread(rng, 1, max(1, min(4096, most))), K=K, N=N, dtype=half, bias=rng.random() < 0.7)
    if kind in ("route", "route_step"):
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _spread(rng, 8, 512 // groups if groups > 1 else 384)
        return dict(kind=kind, T=_spread(rng, 1, 16384), E=E, k=rng.randint(1, 8), score=rng.choice(["softmax", "sigmoid"]),
                    balance=rng.random() < 0.6, groups=groups, top_groups=rng.randint(1, groups), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["fp32", "bf16", "fp16"]), masked=rng.random() < 0.5)
    E, K, I = rng.randint(4, 64), _spread(rng, 256, 4096, 16), _spread(rng, 128, 1536, 16)
    k = rng.randint(1, min(8, E))
    return dict(kind=kind, T=_spread(rng, 1, 1024 if kind == "experts_step" else 2048), E=E, k=k, K=K, I=I, dtype=half,
                padded=rng.random() < 0.5)


def work(case):
    c = case
    blocks = lambda n: -(-n // BLOCK)  # noqa: E731
    if c["kind"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        return {"bytes": 2 * T * K + N * K + 4 * blocks(N) * blocks(K) + 2 * T * N + 2 * N * c["bias"], "flops": 2 * T * N * K}
    if c["kind"] == "linear_step":
        T, K, N = c["T"], c["K"], c["N"]
        return {"bytes": 2 * (2 * T * K + 2 * N * K + 2 * T * N + 2 * N * c["bias"]), "flops": 6 * T * N * K}
    if c["kind"] in ("route", "route_step"):
        size = 4 if c["dtype"] == "fp32" else 2
        step = c["kind"] == "route_step"
        return {"bytes": c["T"] * (c["E"] * size * (2 if step else 1) + c["k"] * (12 if step else 8)), "flops": c["T"] * c["E"] * (8 if step else 4)}
    T, K, I, R = c["T"], c["K"], c["I"], c["T"] * c["k"]
    step = c["kind"] == "experts_step"
    return {"bytes": min(c["E"], R) * 3 * I * K + T * K * 2 * (4 if step else 2) + R * (12 if step else 8), "flops": R * 6 * I * K * (2 if step else 1)}


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _states(gen, T, K, dtype):
    """Hidden states: unit normal values, a few features that carry outliers, tokens of unlike size."""
    x = _normal(gen, T, K) * torch.exp(0.5 * _normal(gen, T, 1))
    x[:, torch.randint(0, K, (max(1, K // 512),), generator=gen, device="cuda")] *= 20.0
    return x.to(dtype)


def _tiles(W):
    """Codes (as bytes) and scales [..., ceil(N/128), ceil(K/128)] of a weight [..., N, K], 128 x 128 each."""
    N, K = W.shape[-2:]
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    P = torch.nn.functional.pad(W, (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(*W.shape[:-2], nb, BLOCK, kb, BLOCK)
    a = P.float().abs().amax(dim=(-3, -1)).clamp_min(FLOOR)
    up = torch.full_like(a, 448.0) / a
    q = (P * up[..., :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(*W.shape[:-2], nb * BLOCK, kb * BLOCK)[..., :N, :K].contiguous(), a * (1.0 / 448.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, s = case, {"case": dict(case)}
    if c["kind"] in ("linear", "linear_step"):
        T, K, N, dtype = c["T"], c["K"], c["N"], DTYPES[c["dtype"]]
        s["x"] = _states(gen, T, K, dtype)
        s["bias"] = _normal(gen, N).to(dtype) if c["bias"] else None
        if c["kind"] == "linear":
            rows = max(BLOCK, (1 << 28) // K // BLOCK * BLOCK)  # quantised in pieces: the widest weight is large
            parts = [_tiles(_normal(gen, min(rows, N - n), K) * 0.02) for n in range(0, N, rows)]
            s["codes"], s["scales"] = (torch.cat(p) for p in zip(*parts))
        else:
            s["weight"] = (_normal(gen, N, K) * 0.02).to(dtype)
            s["dy"] = (_normal(gen, T, N) * torch.exp(_normal(gen, T, 1)) * 1e-2).to(dtype)
            for v in (s["x"], s["weight"], s["bias"]):
                if v is not None:
                    v.requires_grad_(True)
    elif c["kind"] in ("route", "route_step"):
        T, E = c["T"], c["E"]
        logits = (_normal(gen, T, E) + 0.7 * _normal(gen, E)).to(DTYPES[c["dtype"]])
        if c["masked"]:
            dead = torch.rand((T, 1), generator=gen, device="cuda") < 0.1  # tokens of padding
            gone = torch.rand((T, E), generator=gen, device="cuda") < 0.2
            logits.masked_fill_(dead | gone, float("-inf"))
        s["logits"] = logits
        s["balance"] = 0.1 * _normal(gen, E) if c["balance"] else None
        if c["kind"] == "route_step":
            s["dw"] = _normal(gen, T, c["k"])
            logits.requires_grad_(True)
    else:
        T, E, K, I, dtype = c["T"], c["E"], c["K"], c["I"], DTYPES[c["dtype"]]
        s["x"] = _states(gen, T, K, dtype)
        s["codes13"], s["scales13"] = _tiles((_normal(gen, E, 2, I, K) * 0.03).to(dtype))
        s["codes2"], s["scales2"] = _tiles((_normal(gen, E, K, I) * 0.03).to(dtype))
        popular = _normal(gen, T, E) + _normal(gen, E)
        top = torch.sort(popular, dim=1, descending=True, stable=True)
        s["idx"] = top.indices[:, : c["k"]].to(torch.int32).contiguous()
        if c["padded"]:
            s["idx"].masked_fill_(torch.rand((T, 1), generator=gen, device="cuda") < 0.1, -1)
        s["w"] = torch.softmax(top.values[:, : c["k"]], dim=1).contiguous()
        # the longest expert's rows: what the plain form pads to
        s["capacity"] = int(torch.bincount(s["idx"].flatten().long() + 1, minlength=E + 1)[1:].max())
        if c["kind"] == "experts_step":
            s["dy"] = (_normal(gen, T, K) * 1e-2).to(dtype)
            s["x"].requires_grad_(True)
            s["w"].requires_grad_(True)
    return s


# ------------------------------------------------------------------ plain forms
def _rows(v):
    """The values that v [..., K] stands for in blocks of 128 along its last dimension."""
    K = v.shape[-1]
    kb = -(-K // BLOCK)
    p = torch.nn.functional.pad(v.float(), (0, kb * BLOCK - K)).view(*v.shape[:-1], kb, BLOCK)
    a = p.abs().amax(dim=-1, keepdim=True).clamp_min(FLOOR)
    q = (p * (torch.full_like(a, 448.0) / a)).to(torch.float8_e4m3fn).float() * (a * (1.0 / 448.0))
    return q.view(*v.shape[:-1], kb * BLOCK)[..., :K]


def _values(codes, scales):
    """The values that codes [..., N, K] with a scale for each 128 x 128 tile stand for."""
    N, K = codes.shape[-2:]
    full = scales.repeat_interleave(BLOCK, dim=-2)[..., :N, :].repeat_interleave(BLOCK, dim=-1)[..., :K]
    return codes.view(torch.float8_e4m3fn).float() * full


def _plain_linear(s):
    y = _rows(s["x"]) @ _values(s["codes"], s["scales"]).mT
    return (y if s["bias"] is None else y + s["bias"].float()).to(s["x"].dtype)


def _plain_linear_step(s):
    x, w, dy, dtype = s["x"], s["weight"], s["dy"], s["x"].dtype
    W = _values(*_tiles(w))
    y = _rows(x) @ W.mT
    if s["bias"] is not None:
        y = y + s["bias"].float()
    dx = _rows(dy) @ W
    dw = _values(*_tiles(dy)).mT @ _values(*_tiles(x))
    db = None if s["bias"] is None else dy.float().sum(dim=0).to(dtype)
    return y.to(dtype), dx.to(dtype), dw.to(dtype), db


def _plain_route(s):
    """Weights and indices; scores and sums in 64 bits, since near-equal scores decide the order."""
    c, x = s["case"], s["logits"].double()
    T, E, k = c["T"], c["E"], c["k"]
    live = x > float("-inf")
    p = torch.softmax(x, dim=1) if c["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-x))
    p = torch.where(live, p, 0.0)
    key = torch.where(live, p if s["balance"] is None else p + s["balance"].double(), float("-inf"))
    if c["groups"] > 1:
        G = c["groups"]
        best = torch.sort(key.view(T, G, E // G), dim=2, descending=True, stable=True).values
        best = best[:, :, : 1 if s["balance"] is None else 2]
        total = torch.where(best > float("-inf"), best, 0.0).sum(dim=2)
        total = torch.where(best[:, :, 0] > float("-inf"), total, float("-inf"))
        order = torch.sort(total, dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=x.device).scatter(1, order, True)
        key = torch.where(kept.repeat_interleave(E // G, dim=1), key, float("-inf"))
    top = torch.sort(key, dim=1, descending=True, stable=True)
    idx, found = top.indices[:, :k], top.values[:, :k] > float("-inf")
    picked = torch.where(found, p.gather(1, idx), 0.0)
    total = picked.sum(dim=1, keepdim=True)
    w = torch.where(total > 0, picked / total, 0.0) if c["renorm"] else picked
    return p, picked, total, idx, found, w * c["scale"]


def _plain_route_step(s):
    c = s["case"]
    p, picked, total, idx, found, w = _plain_route(s)
    g = torch.where(found, s["dw"].double(), 0.0) * c["scale"]
    if c["renorm"]:
        g = torch.where(total > 0, (g - (g * picked).sum(dim=1, keepdim=True) / total) / total, 0.0)
    ds = torch.zeros_like(p).scatter_add(1, idx, torch.where(found, g, 0.0))
    if c["score"] == "softmax":
        dx = p * (ds - (ds * p).sum(dim=1, keepdim=True))
    else:
        dx = ds * p * (1.0 - p)
    return w.float(), torch.where(found, idx, -1).int(), dx.to(s["logits"].dtype)


def _places(s):
    """For each (token, choice): its expert, its row among that expert's rows, and whether it has one."""
    c = s["case"]
    e = s["idx"].flatten().long()
    there = e >= 0
    order = torch.sort(e, stable=True).indices
    ranked = torch.empty_like(order).scatter_(0, order, torch.arange(len(e), device=e.device))
    first = (~there).sum() + torch.cumsum(torch.bincount(e + 1, minlength=c["E"] + 1)[1:], 0)
    first = torch.cat([(~there).sum()[None], first])[:-1]
    e = e.clamp_min(0)
    return e, torch.where(there, ranked - first[e], s["capacity"]), there


def _plain_experts(s, step=False):
    """Few rows: each with its own expert's weights. Many: every expert's rows, padded to the longest."""
    c, dtype = s["case"], s["x"].dtype
    T, E, k, K, I = c["T"], c["E"], c["k"], c["K"], c["I"]
    x = _rows(s["x"])
    source = torch.arange(T * k, device=x.device) // k
    e, place, there = _places(s)
    W13, W2 = (s["codes13"], s["scales13"]), (s["codes2"], s["scales2"])
    if T * k <= E:
        W13, W2 = (tuple(v[e] for v in W) for W in (W13, W2))
        lay = lambda rows: rows[:, None]  # noqa: E731
        back = lambda out: out[:, 0]  # noqa: E731
    else:
        def lay(rows):
            out = torch.zeros((E, s["capacity"] + 1, rows.shape[1]), device=x.device)
            out[e, place] = torch.where(there[:, None], rows, 0.0)
            return out

        def back(out):
            return out[e, place]
    W13, W2 = _values(*W13), _values(*W2)
    gu = lay(x[source])[:, None] @ W13.mT
    g, u = gu[:, 0], gu[:, 1]
    gate = g / (1.0 + torch.exp(-g))
    h = gate * u
    w = torch.where(there, s["w"].flatten(), 0.0)
    out = back(_rows(h) @ W2.mT) * w[:, None]
    y = torch.where(there[:, None], out, 0.0).view(T, k, K).sum(dim=1).to(dtype)
    if not step:
        return y
    dh = lay(_rows(s["dy"])[source]) @ W2
    dw = torch.where(there, back((dh * h).sum(dim=2, keepdim=True))[:, 0], 0.0).view(T, k)
    dh = dh * lay(w[:, None])
    sig = 1.0 / (1.0 + torch.exp(-g))
    dg, du = dh * u * sig * (1.0 + g * (1.0 - sig)), dh * gate
    dx = back(_rows(dg) @ W13[:, 0] + _rows(du) @ W13[:, 1])
    return y, torch.where(there[:, None], dx, 0.0).view(T, k, K).sum(dim=1).to(dtype), dw


def run(state):
    s, c = state, state["case"]
    kind = c["kind"]
    if own:
        from bit_matmul_decomposition_b200 import block, experts
        if kind == "linear":
            return block.linear_block_fp8(s["x"], s["codes"], s["scales"], s["bias"])
        if kind == "linear_step":
            y = block.linear_block_fp8_train(s["x"], s["weight"], s["bias"])
            wanted = [v for v in (s["x"], s["weight"], s["bias"]) if v is not None]
            grads = torch.autograd.grad(y, wanted, s["dy"])
            return [y.detach(), *grads]
        if kind in ("route", "route_step"):
            w, idx = experts.route_experts(s["logits"], c["k"], s["balance"], score=c["score"], n_groups=c["groups"],
                                           top_groups=c["top_groups"], renormalize=c["renorm"], scale=c["scale"])
            if kind == "route":
                return w, idx
            return w.detach(), idx, torch.autograd.grad(w, s["logits"], s["dw"])[0]
        y = experts.experts_block_fp8(s["x"], s["idx"], s["w"], s["codes13"], s["scales13"], s["codes2"], s["scales2"])
        if kind == "experts":
            return y
        return [y.detach(), *torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])]
    with torch.no_grad():
        if kind == "linear":
            return _plain_linear(s)
        if kind == "linear_step":
            return [v for v in _plain_linear_step(s) if v is not None]
        if kind == "route":
            _, _, _, idx, found, w = _plain_route(s)
            return w.float(), torch.where(found, idx, -1).int()
        if kind == "route_step":
            return _plain_route_step(s)
        return _plain_experts(s, step=kind == "experts_step")


# ------------------------------------------------------------------ values in 64 bits
def _nearest(v):
    """e4m3 value nearest to v (ties to even): 4 significant bits, steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.frexp(v)[1].clamp_min(-5).double() - 4)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _quantised(v, across):
    """Values of v [..., R, C] in blocks of 128 columns, and of `across` rows (1 or 128)."""
    v = v.double()
    R, C = v.shape[-2:]
    out = torch.empty_like(v)
    for r0 in range(0, R, max(across, 8192)):
        for c0 in range(0, C, BLOCK):
            t = v[..., r0: r0 + max(across, 8192), c0: c0 + BLOCK]
            m = t.abs().amax(dim=-1, keepdim=True)
            if across > 1:
                n = -(-t.shape[-2] // across)
                m = torch.stack([m[..., i * across: (i + 1) * across, :].amax(dim=-2) for i in range(n)], dim=-2)
                m = m.repeat_interleave(across, dim=-2)[..., : t.shape[-2], :]
            m = m.clamp_min(FLOOR)
            up = (448.0 / m).float().double()
            down = (m * torch.tensor(1.0 / 448.0).item()).float().double()  # 1 / 448 as 32 bits hold it
            out[..., r0: r0 + max(across, 8192), c0: c0 + BLOCK] = _nearest((t * up).float().double()) * down
    return out


def _stands_for(codes, scales):
    out = codes.view(torch.float8_e4m3fn).double()
    for n in range(scales.shape[-2]):
        out[..., n * BLOCK: (n + 1) * BLOCK, :] *= scales[..., n, :].double().repeat_interleave(BLOCK, dim=-1)[..., None, : out.shape[-1]]
    return out


def _exact_route(s):
    c = s["case"]
    x = s["logits"].detach().double()
    if c["score"] == "softmax":
        top = x.amax(dim=1, keepdim=True)
        z = torch.exp(x - torch.where(torch.isfinite(top), top, 0.0))
        p = z / z.sum(dim=1, keepdim=True).clamp_min(1e-300)
    else:
        p = torch.sigmoid(x)
    value = p.clone() if s["balance"] is None else p + s["balance"].double()
    value[torch.isinf(x)] = -1e30
    if c["groups"] > 1:
        size = c["E"] // c["groups"]
        byg = value.view(c["T"], c["groups"], size)
        most = 1 if s["balance"] is None else min(2, size)
        m = byg.topk(most, dim=2).values
        rank = (m * (m > -1e29)).sum(dim=2) + torch.where(m[..., 0] > -1e29, 0.0, -1e30)
        ahead = (rank[:, None, :] > rank[:, :, None]).sum(dim=2)
        same = (rank[:, None, :] == rank[:, :, None]).double().tril(-1).sum(dim=2)
        byg[(ahead + same) >= c["top_groups"]] = -1e30
    idx = torch.empty((c["T"], c["k"]), dtype=torch.long, device=x.device)
    ok = torch.empty((c["T"], c["k"]), dtype=torch.bool, device=x.device)
    left = value.clone()
    for j in range(c["k"]):
        m = left.amax(dim=1, keepdim=True)
        idx[:, j] = (left == m).double().argmax(dim=1)
        ok[:, j] = m[:, 0] > -1e29
        left.scatter_(1, idx[:, j: j + 1], -2e30)
    ps = p.gather(1, idx) * ok
    S = ps.sum(dim=1, keepdim=True)
    w = (ps / S.clamp_min(1e-300) if c["renorm"] else ps) * c["scale"]
    return p, ps, S, idx, ok, w


def exact(case, seed):
    c, s = case, prepare(case, seed)
    with torch.no_grad():
        if c["kind"] == "linear":
            x = _quantised(s["x"], 1)
            rows = max(BLOCK, (1 << 29) // c["K"] // BLOCK * BLOCK)
            y = torch.cat([x @ _stands_for(s["codes"][n: n + rows], s["scales"][n // BLOCK: (n + rows) // BLOCK]).T
                           for n in range(0, c["N"], rows)], dim=1)
            return y if s["bias"] is None else y + s["bias"].double()
        if c["kind"] == "linear_step":
            W, dy = _quantised(s["weight"], BLOCK), s["dy"]
            y = _quantised(s["x"], 1) @ W.T
            got = [y if s["bias"] is None else y + s["bias"].double(), _quantised(dy, 1) @ W,
                   _quantised(dy, BLOCK).T @ _quantised(s["x"], BLOCK)]
            return got if s["bias"] is None else got + [dy.double().sum(dim=0)]
        if c["kind"] in ("route", "route_step"):
            p, ps, S, idx, ok, w = _exact_route(s)
            if c["kind"] == "route":
                return w, None
            g = s["dw"].double() * ok * c["scale"]
            if c["renorm"]:
                S = S.clamp_min(1e-300)
                g = (g / S - (g * ps).sum(dim=1, keepdim=True) / (S * S)) * ok
            ds = torch.zeros_like(p).scatter_add_(1, idx, g)
            dx = p * ds - p * (ds * p).sum(dim=1, keepdim=True) if c["score"] == "softmax" else ds * (p - p * p)
            return w, None, dx
        x, w = _quantised(s["x"], 1), s["w"].double()
        step = c["kind"] == "experts_step"
        y, dx, dw = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(w)
        dy = _quantised(s["dy"], 1) if step else None
        for e in range(c["E"]):  # expert by expert
            t, j = torch.nonzero(s["idx"] == e, as_tuple=True)
            if len(t) == 0:
                continue
            W1, W3 = _stands_for(s["codes13"][e], s["scales13"][e])
            W2 = _stands_for(s["codes2"][e], s["scales2"][e])
            g, u = x[t] @ W1.T, x[t] @ W3.T
            h = g * torch.sigmoid(g) * u
            y.index_add_(0, t, (_quantised(h, 1) @ W2.T) * w[t, j][:, None])
            if step:
                dh = dy[t] @ W2
                dw[t, j] = (dh * h).sum(dim=1)
                dh = dh * w[t, j][:, None]
                sg = torch.sigmoid(g)
                dx.index_add_(0, t, _quantised(dh * u * (sg + g * sg * (1 - sg)), 1) @ W1 + _quantised(dh * g * sg, 1) @ W3)
        return [y, dx, dw] if step else y
