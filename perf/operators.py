"""The operators around the FP8 path of a mixture-of-experts layer, as measurable cases:

  router   which experts a token goes to: scores from the logits, top-k, routing weights,
           per-expert counts and the balance loss, with the gradient of both;
  stash    SwiGLU forward that keeps gate and up for the backward pass as 8-bit codes;
  bwd      SwiGLU backward from those codes (BF16 gradients, or E4M3 ones);
  linear   rows times 4-bit microscaled weights: quantisation of the rows and the product;
  experts  the same for routed tokens: permute, quantisation and the experts' products.

`own` false: plain torch operations; `own` true: the calls of scaling_aware_transpose_b200.
FP8 codes are returned as the float8 values they stand for, with their scales beside them.
"""
import math

import torch

own = False
DEV = "cuda"
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of an E2M1 code


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # One token of a decode step: 32 experts, top-8 (the repository's MoE workload).
        dict(name="router_token", op="router", tokens=1, experts=32, topk=8, dtype="bf16", sigmoid=False, renorm=True,
             bias=False, mask=False, train=False),
        # The MoE workload's training step, gradient included.
        dict(name="router_train", op="router", tokens=16384, experts=32, topk=8, dtype="bf16", sigmoid=False,
             renorm=True, bias=False, mask=False, train=True),
        # Many experts, sigmoid scores with a selection bias, fp32 logits, a ragged batch.
        dict(name="router_wide", op="router", tokens=50021, experts=256, topk=8, dtype="fp32", sigmoid=True,
             renorm=True, bias=True, mask=False, train=True),
        # A padded batch with an odd number of experts and some experts switched off.
        dict(name="router_odd", op="router", tokens=4099, experts=60, topk=6, dtype="fp32", sigmoid=False,
             renorm=False, bias=False, mask=True, train=True),
        # SwiGLU workload: rows of one training step's experts.
        dict(name="stash_step", op="stash", rows=32768, cols=2048, weights=True),
        # A handful of rows, as one token's experts.
        dict(name="stash_few", op="stash", rows=8, cols=2048, weights=True),
        dict(name="bwd_step", op="bwd", rows=32768, cols=2048, weights=True, fp8=False),
        # The MoE workload's padded rows, gradients in FP8 for the FP8 products.
        dict(name="bwd_fp8", op="bwd", rows=133120, cols=2048, weights=True, fp8=True),
        # One token through one projection: the weights' bytes bound it.
        dict(name="linear_token", op="linear", m=1, n=4096, k=7168),
        # Odd sizes on every side.
        dict(name="linear_odd", op="linear", m=1003, n=2050, k=1408),
        # A prompt's rows through a full projection.
        dict(name="linear_prompt", op="linear", m=8192, n=4096, k=7168),
        # Routed tokens through 32 experts' first projection.
        dict(name="experts", op="experts", tokens=4096, experts=32, topk=8, n=2048, k=7168),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "router", "stash", "bwd", "bwd", "linear", "linear", "experts"])
    if op == "router":
        experts = _log(rng, 8, 512)
        tokens = _log(rng, 1, 65536)
        sigmoid = rng.random() < 0.5
        return dict(op=op, tokens=tokens, experts=experts, topk=rng.randint(1, 8), dtype=rng.choice(["bf16", "fp32"]),
                    sigmoid=sigmoid, renorm=rng.random() < 0.6, bias=sigmoid and rng.random() < 0.7,
                    mask=rng.random() < 0.4, train=rng.random() < 0.7)
    if op in ("stash", "bwd"):
        cols = 128 * rng.randint(1, 32)
        rows = min(_log(rng, 1, 131072), 133120 * 2048 // cols)
        c = dict(op=op, rows=rows, cols=cols, weights=rng.random() < 0.6)
        if op == "bwd":
            c["fp8"] = rng.random() < 0.5
        return c
    if op == "linear":
        return dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 64, 4096), k=128 * rng.randint(1, 56))
    return dict(op=op, tokens=_log(rng, 1, 4096), experts=rng.choice([4, 8, 16, 32]), topk=rng.randint(1, 4),
                n=128 * rng.randint(1, 16), k=128 * rng.randint(1, 56))


def work(case):
    c = case
    if c["op"] == "router":
        T, E, K = c["tokens"], c["experts"], c["topk"]
        el = 2 if c["dtype"] == "bf16" else 4
        b = T * E * el + 8 * T * K + (T if c["mask"] else 0) + (4 * E if c["bias"] else 0) + 8 * E + 4
        f = T * E * 6
        if c["train"]:  # logits in, gradient out, ids and weight gradients in
            b += 2 * T * E * el + 8 * T * K + (T if c["mask"] else 0) + 4 * E
            f += T * E * 12
        return {"bytes": b, "flops": f}
    if c["op"] in ("stash", "bwd"):
        n, t = c["rows"] * c["cols"], c["rows"] * c["cols"] // 128
        w = 4 * c["rows"] if c["weights"] else 0
        if c["op"] == "stash":
            return {"bytes": 7 * n + 3 * t + w, "flops": 10 * n}
        return {"bytes": (7 * n + 5 * t if c["fp8"] else 8 * n + 2 * t) + 2 * w, "flops": 16 * n}
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": 2 * m * k + n * k // 2 + n * k // 32 + 2 * m * n, "flops": 2 * m * n * k}
    T, E, K, n, k = c["tokens"], c["experts"], c["topk"], c["n"], c["k"]
    hit = min(E, T * K)
    return {"bytes": 2 * T * k + 4 * T * K + hit * (n * k // 2 + n * k // 32) + 2 * T * K * n, "flops": 2 * T * K * n * k}


# ------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    s = {"case": dict(c)}
    if c["op"] == "router":
        T, E, K = c["tokens"], c["experts"], c["topk"]
        # some experts are more popular than others
        logits = randn(T, E) * 1.2 - 0.6 * torch.log1p(torch.arange(E, device=DEV).float())[torch.randperm(E, generator=g, device=DEV)]
        s["mask"] = s["bias"] = None
        if c["mask"]:
            s["mask"] = (rand(T) >= 0.1).to(torch.uint8)
            logits[:, E - 2] = -math.inf  # an expert that is switched off
            logits[s["mask"] == 0] = math.nan  # what padding rows may hold
        if c["bias"]:
            s["bias"] = randn(E) * 0.1
        s["logits"] = logits.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
        s["grad_weights"] = randn(T, K)
        s["grad_loss"] = rand(1) + 0.5
        return s
    if c["op"] == "stash":
        f = torch.exp(randn(c["rows"], 1))
        s["gate"] = (randn(c["rows"], c["cols"]) * f).to(torch.bfloat16)
        s["up"] = (randn(c["rows"], c["cols"]) * f).to(torch.bfloat16)
        s["w"] = rand(c["rows"]) if c["weights"] else None
        return s
    if c["op"] == "bwd":
        f = torch.exp(randn(c["rows"], 1))
        s["gq"], s["gsf"] = _quant8(randn(c["rows"], c["cols"]) * f)
        s["uq"], s["usf"] = _quant8(randn(c["rows"], c["cols"]) * f)
        s["dy"] = (randn(c["rows"], c["cols"]) * 1e-3).to(torch.bfloat16)
        s["w"] = rand(c["rows"]) if c["weights"] else None
        return s
    k, n = c["k"], c["n"]
    groups = c["experts"] if c["op"] == "experts" else 1
    w = randn(groups * n, k) * torch.exp(0.5 * randn(groups * n, 1)) / math.sqrt(k)
    s["wq"], s["wsf"] = _codes4(w)  # packed codes [groups*n, k/2], scale bytes [groups*n, k/32]
    del w
    rows = c["tokens"] if c["op"] == "experts" else c["m"]
    s["x"] = (randn(rows, k) * torch.exp(randn(rows, 1))).to(torch.bfloat16)
    if c["op"] == "experts":
        E, K = c["experts"], c["topk"]
        score = randn(rows, E) - 1.1 * torch.log(1.0 + torch.arange(E, device=DEV))  # Zipf(1.1) popularity
        s["idx"] = torch.topk(score, K, dim=1).indices.to(torch.int32)
        s["out"] = torch.zeros((rows * K + E * 127, n), dtype=torch.bfloat16, device=DEV)  # rows past the last group stay
    return s


# ------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        import scaling_aware_transpose_b200 as sat
        return _own(s, c, sat)
    if c["op"] == "router":
        return _plain_router(s, c)
    if c["op"] == "stash":
        y = _silu(s["gate"].float()) * s["up"].float()
        if s["w"] is not None:
            y = y * s["w"][:, None]
        return [*_values8(*_quant8(y)), *_values8(*_quant8(s["gate"].float())), *_values8(*_quant8(s["up"].float()))]
    if c["op"] == "bwd":
        return _plain_bwd(s, c)
    if c["op"] == "linear":
        return torch.matmul(_decode4(*_codes4(s["x"].float())), _decode4(s["wq"], s["wsf"]).t()).to(torch.bfloat16)
    return _plain_experts(s, c)


def _own(s, c, sat):
    if c["op"] == "router":
        o = dict(sigmoid=c["sigmoid"], renormalize=c["renorm"], token_mask=s["mask"], scale=1.0)
        idx, w, counts, sums, loss = sat.router_topk(s["logits"], c["topk"], bias=s["bias"], balance=c["train"],
                                                     loss_coef=0.01, **o)
        if not c["train"]:
            return [idx, w]
        grad = sat.router_topk_bwd(s["logits"], idx, s["grad_weights"], counts=counts, grad_loss=s["grad_loss"],
                                   loss_coef=0.01, **o)
        return [idx, w, counts, sums, loss, grad]
    if c["op"] == "stash":
        q, sf, gq, gsf, uq, usf = sat.swiglu_quant_stash(s["gate"], s["up"], row_weights=s["w"])
        return [*_values8(q, sf), *_values8(gq, gsf), *_values8(uq, usf)]
    if c["op"] == "bwd":
        if not c["fp8"]:
            dg, du, dw = sat.swiglu_bwd(s["gq"], s["gsf"], s["uq"], s["usf"], s["dy"], row_weights=s["w"])
            return [dg, du] if dw is None else [dg, du, dw]
        dgq, dgsf, duq, dusf, yq, ysf, dw = sat.swiglu_bwd_quant(s["gq"], s["gsf"], s["uq"], s["usf"], s["dy"],
                                                                 row_weights=s["w"])
        out = [*_values8(dgq, dgsf), *_values8(duq, dusf), *_values8(yq, ysf)]
        return out if dw is None else [*out, dw]
    if "wsf_tiled" not in s:  # laid out once, when the weights are loaded
        s["wsf_tiled"] = sat.mxfp4_tile_scales(s["wsf"])
    if c["op"] == "linear":
        xq, xsf = sat.quantize_rowwise_mxfp4(s["x"])
        return sat.matmul_mxfp4(xq, xsf, s["wq"], s["wsf_tiled"])
    q, sf, off, _ = sat.permute_pad_mxfp4(s["x"], s["idx"], c["experts"], 128)
    return sat.matmul_mxfp4(q, sf, s["wq"], s["wsf_tiled"], group_offsets=off, out=s["out"])


# ------------------------------------------------------------------------------- plain forms
def _silu(g):
    return g / (1 + torch.exp(-g))


def _quant8(x):
    """E4M3 codes with one power-of-two scale per 1x128 tile: S = 2^e, the least e with amax <= 448 * 2^e."""
    r, c = x.shape
    t = x.view(r, c // 128, 128)
    amax = t.abs().amax(-1)
    m, p = torch.frexp(amax)  # amax = m * 2^p, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(amax == 0, 0, p - 9 + (m > 0.875).int()).clamp_min(-127)
    q = torch.ldexp(t, -e[..., None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(r, c), (e + 127).to(torch.uint8)


def _values8(q, sf):
    return q.view(torch.float8_e4m3fn), sf.view(torch.float8_e8m0fnu)


def _decode8(q, sf):
    r, c = q.shape
    return torch.ldexp(q.view(torch.float8_e4m3fn).float().view(r, c // 128, 128), sf.int()[..., None] - 127).view(r, c)


def _codes4(x):
    """E2M1 codes, two to a byte (even column low), one power-of-two scale per 1x32 tile: the least e with amax <= 6 * 2^e."""
    r, c = x.shape
    t = x.view(r, c // 32, 32)
    amax = t.abs().amax(-1)
    m, p = torch.frexp(amax)  # 6 = 0.75 * 2^3
    e = torch.where(amax == 0, 0, p - 3 + (m > 0.75).int()).clamp_min(-127)
    v = torch.ldexp(t, -e[..., None])
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))  # ties to even
    code = (code + 8 * torch.signbit(v)).to(torch.uint8).view(r, c // 2, 2)
    return code[..., 0] + 16 * code[..., 1], (e + 127).to(torch.uint8)


def _decode4(q, sf):
    r, h = q.shape
    codes = torch.stack([q & 15, q >> 4], -1).int()
    mag = torch.tensor(GRID, device=q.device)[codes & 7]
    v = torch.where(codes >= 8, -mag, mag).view(r, h // 16, 32)
    return torch.ldexp(v, sf.int()[..., None] - 127).view(r, 2 * h)


def _plain_router(s, c):
    T, E, K = c["tokens"], c["experts"], c["topk"]
    l = s["logits"].float()
    l = torch.where(torch.isnan(l), -math.inf, l)
    live = torch.ones(T, dtype=torch.bool, device=l.device) if s["mask"] is None else s["mask"] != 0
    if c["sigmoid"]:
        p = 1 / (1 + torch.exp(-l))
        total = p.sum(1, keepdim=True) + 1e-20
        key = 1 / (1 + torch.exp(-l.double())) + s["bias"].double() if c["bias"] else l
    else:
        m = l.amax(1, keepdim=True)
        x = torch.exp(l - torch.where(torch.isinf(m), 0.0, m))
        z = x.sum(1, keepdim=True)
        p = x / torch.where(z == 0, 1.0, z)
        key = l
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K]
    ps = torch.gather(p, 1, idx)
    norm = ps.sum(1, keepdim=True) + 1e-20 if c["renorm"] else torch.ones_like(ps[:, :1])
    w = torch.where(live[:, None], ps / norm, 0.0)
    if not c["train"]:
        return [idx.to(torch.int32), w]
    counts = torch.zeros(E, dtype=torch.int64, device=l.device)
    counts.scatter_add_(0, idx.reshape(-1), live[:, None].expand(T, K).reshape(-1).long())
    share = p / total if c["sigmoid"] else p
    sums = torch.where(live[:, None], share, 0.0).double().sum(0).float()
    C = counts.sum().double()
    coef = torch.where(C > 0, 0.01 * E * K / (C * C).clamp_min(1), 0.0)
    loss = (coef * (counts.double() * sums.double()).sum()).float().view(1)
    # gradient
    d = torch.zeros_like(p)
    dw = s["grad_weights"]
    back = dw / norm - ((dw * ps).sum(1, keepdim=True) / (norm * norm) if c["renorm"] else 0.0)
    d.scatter_(1, idx, back)
    ge = (s["grad_loss"].double() * coef * counts.double()).float()
    if c["sigmoid"]:
        d = d + (ge - (ge * share).sum(1, keepdim=True)) / total
        grad = d * p * (1 - p)
    else:
        d = d + ge
        grad = p * (d - (d * p).sum(1, keepdim=True))
    grad = torch.where(live[:, None], grad, 0.0)
    return [idx.to(torch.int32), w, counts.to(torch.int32), sums, loss, grad.to(s["logits"].dtype)]


def _plain_bwd(s, c):
    g, u = _decode8(s["gq"], s["gsf"]), _decode8(s["uq"], s["usf"])
    dy = s["dy"].float()
    sig = 1 / (1 + torch.exp(-g))
    y = g * sig * u
    dw = None
    if s["w"] is not None:
        dw = (dy.double() * y.double()).sum(1).float()
        y = y * s["w"][:, None]
        dy = dy * s["w"][:, None]
    dg = dy * u * sig * (1 + g * (1 - sig))
    du = dy * g * sig
    if c["fp8"]:
        out = [*_values8(*_quant8(dg)), *_values8(*_quant8(du)), *_values8(*_quant8(y))]
    else:
        out = [dg.to(torch.bfloat16), du.to(torch.bfloat16)]
    return out if dw is None else [*out, dw]


def _slots(idx, E):
    """Destination row of each (token, slot) pair and the group ends, groups padded to 128 rows."""
    e = idx.reshape(-1).long()
    order = torch.sort(e, stable=True).indices
    counts = torch.zeros(E, dtype=torch.int64, device=e.device).scatter_add_(0, e, torch.ones_like(e))
    ends = torch.cumsum((counts + 127) // 128 * 128, 0)
    starts = ends - (counts + 127) // 128 * 128
    rank = torch.arange(e.numel(), device=e.device) - (torch.cumsum(counts, 0) - counts)[e[order]]
    row = torch.empty_like(e)
    row[order] = starts[e[order]] + rank
    return row, ends


def _plain_experts(s, c):
    E, K, n, k = c["experts"], c["topk"], c["n"], c["k"]
    row, ends = _slots(s["idx"], E)
    blocks = (s["out"].shape[0] + 127) // 128
    x = torch.zeros((blocks * 128, k), device=row.device)
    x[row] = torch.repeat_interleave(_decode4(*_codes4(s["x"].float())), K, 0)
    w = _decode4(s["wq"], s["wsf"]).view(E, n, k)
    expert = torch.bucketize(torch.arange(blocks, device=row.device) * 128, ends, right=True).clamp_max(E - 1)
    y = torch.bmm(x.view(blocks, 128, k), w[expert].transpose(1, 2)).view(blocks * 128, n)
    out = s["out"]
    out.copy_(y[:out.shape[0]])
    return out


# ------------------------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "router":
        return _exact_router(s, c)
    if c["op"] == "stash":
        g, u = s["gate"].double(), s["up"].double()
        y = g * torch.sigmoid(g) * u * (1.0 if s["w"] is None else s["w"].double()[:, None])
        return [_over_scale(y), None, _over_scale(g), None, _over_scale(u), None]
    if c["op"] == "bwd":
        g, u = (s[q].view(torch.float8_e4m3fn).double() * torch.exp2(s[f].double() - 127).repeat_interleave(128, 1)
                for q, f in (("gq", "gsf"), ("uq", "usf")))
        dy = s["dy"].double()
        act = g * torch.sigmoid(g)
        slope = torch.sigmoid(g) + act * torch.sigmoid(-g)
        w = torch.ones_like(dy[:, :1]) if s["w"] is None else s["w"].double()[:, None]
        dg, du, y = w * dy * u * slope, w * dy * act, w * act * u
        out = [_over_scale(dg), None, _over_scale(du), None, _over_scale(y), None] if c["fp8"] else [dg, du]
        return out if s["w"] is None else [*out, (dy * act * u).sum(1)]
    xr = _round4(s["x"].double())
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=DEV)
    wd = torch.stack((grid[(s["wq"] % 16).long()], grid[(s["wq"] // 16).long()]), 2).flatten(1)
    wd = wd * torch.exp2(s["wsf"].double() - 127).repeat_interleave(32, 1)
    if c["op"] == "linear":
        return xr @ wd.T
    E, K, n = c["experts"], c["topk"], c["n"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for e in range(E):  # each expert's tokens in order, then padding to 128 rows
        tok = (s["idx"] == e).nonzero()[:, 0]
        out[at:at + tok.numel()] = xr[tok] @ wd[e * n:(e + 1) * n].T
        at += -(-tok.numel() // 128) * 128
    return out


def _over_scale(v):
    """Each value over its tile's scale: what an E4M3 code stands for, before it is rounded."""
    t = v.unflatten(1, (-1, 128))
    top = t.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2(top / 448)).clamp(-127, 127)
    e = torch.where(top > 448 * torch.exp2(e), e + 1, torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e))
    return (t / torch.exp2(torch.where(top == 0, 0.0, e))).flatten(1)


def _round4(v):
    """Rows rounded to E2M1 with a power-of-two scale per 32 columns, in 64 bits."""
    t = v.unflatten(1, (-1, 32))
    top = t.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2(top / 6))
    e = torch.where(top > 6 * torch.exp2(e), e + 1, torch.where(top <= 6 * torch.exp2(e - 1), e - 1, e))
    scale = torch.exp2(torch.where(top == 0, 0.0, e).clamp(-127, 127))
    t = t / scale
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(1.0))) - 1)
    return (torch.round(t / step) * step * scale).flatten(1)


def _exact_router(s, c):
    T, E, K = c["tokens"], c["experts"], c["topk"]
    l = torch.nan_to_num(s["logits"].double(), nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    live = torch.ones((T, 1), dtype=torch.float64, device=DEV) if s["mask"] is None else (s["mask"] > 0).double()[:, None]
    if c["sigmoid"]:
        score = torch.sigmoid(l)
        share = score / (score.sum(1, keepdim=True) + 1e-20)
        rank_by = score + s["bias"].double() if c["bias"] else l
    else:
        score = share = torch.nan_to_num(torch.softmax(l, 1))
        rank_by = l
    idx = torch.argsort(-rank_by, dim=1, stable=True)[:, :K]
    hot = torch.zeros_like(score).scatter_(1, idx, 1.0)
    top = (score * hot).sum(1, keepdim=True) + 1e-20 if c["renorm"] else torch.ones_like(live)
    w = live * score.gather(1, idx) / top
    if not c["train"]:
        return [idx.int(), w]
    counts = (hot * live).sum(0)
    sums = (share * live).sum(0)
    N = live.sum().clamp_min(1)
    loss = 0.01 * E * ((counts / (N * K)) * (sums / N)).sum()
    up = torch.zeros_like(score).scatter_(1, idx, s["grad_weights"].double())
    d = hot * (up - ((up * score).sum(1, keepdim=True) / top if c["renorm"] else 0.0)) / top
    pull = s["grad_loss"].double() * 0.01 * E * counts / (N * K) / N
    if c["sigmoid"]:
        d = d + (pull - share @ pull[:, None]) / (score.sum(1, keepdim=True) + 1e-20)
        grad = d * score * torch.sigmoid(-l)
    else:
        d = d + pull
        grad = score * d - score * (score * d).sum(1, keepdim=True)
    return [idx.int(), w, counts.int(), sums, loss.view(1), live * grad]
