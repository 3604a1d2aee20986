"""Plain 64-bit forms of the router, the SwiGLU backward and the 4-bit quantization, from
their definitions (numpy float64 on the host), and the error bounds of their fp32 kernels."""
import numpy as np

U = 2.0 ** -24      # half a step of fp32, relative
U_BF16 = 2.0 ** -8  # half a step of BF16, relative


def clean(logits):
    l = np.asarray(logits, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    return np.minimum(l, np.finfo(np.float32).max)


def router(logits, topk, sigmoid=False, renorm=True, bias=None, mask=None, scale=1.0, loss_coef=1.0):
    """dict(idx, weights, counts, sums, loss, p, h, P) in float64."""
    l = clean(logits)
    T, E = l.shape
    live = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    with np.errstate(all="ignore"):
        if sigmoid:
            p = 1.0 / (1.0 + np.exp(-l))
            h = p / (p.sum(1, keepdims=True) + 1e-20)
        else:
            m = l.max(1, keepdims=True)
            x = np.exp(l - np.where(np.isinf(m), 0.0, m))
            z = x.sum(1, keepdims=True)
            p = x / np.where(z == 0, 1.0, z)
            h = p
    key = p + np.asarray(bias, np.float64) if bias is not None else l
    key = np.where(np.isnan(key), -np.inf, key)
    if bias is not None:  # experts that are off come behind all others, by the bias among themselves
        order = np.lexsort((-key, np.isneginf(l)), axis=1)
        key = np.empty_like(key)
        np.put_along_axis(key, order, np.broadcast_to(-np.arange(E, dtype=np.float64), (T, E)), 1)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :topk]
    pk = np.take_along_axis(p, idx, 1)
    P = pk.sum(1, keepdims=True) + 1e-20 if renorm else np.ones((T, 1))
    w = np.where(live[:, None], scale * pk / P, 0.0)
    counts = np.bincount(idx[live].reshape(-1), minlength=E)
    sums = h[live].sum(0)
    C = float(counts.sum())
    coef = loss_coef * E * topk / C ** 2 if C else 0.0
    return dict(idx=idx, weights=w, counts=counts, sums=sums, loss=coef * float((counts * sums).sum()), p=p, h=h, P=P,
                live=live, coef=coef)


def router_bwd(logits, idx, grad_weights, counts, grad_loss, sigmoid=False, renorm=True, mask=None, scale=1.0,
               loss_coef=1.0):
    """(gradient of the logits, a magnitude bound of what was added up to form it)."""
    T, E = np.asarray(logits).shape
    K = idx.shape[1]
    r = router(logits, K, sigmoid, renorm, None, mask, scale, loss_coef)
    p, h = r["p"], r["h"]
    pk = np.take_along_axis(p, idx, 1)
    P = pk.sum(1, keepdims=True) + 1e-20 if renorm else np.ones((T, 1))
    d = np.zeros((T, E))
    A = np.zeros((T, E))
    if grad_weights is not None:
        gw = np.asarray(grad_weights, np.float64)
        mean = (gw * pk).sum(1, keepdims=True) / P if renorm else 0.0
        mean_abs = (np.abs(gw) * pk).sum(1, keepdims=True) / P if renorm else 0.0
        t = np.arange(T)[:, None].repeat(K, 1)
        np.add.at(d, (t, idx), scale * (gw - mean) / P)
        np.add.at(A, (t, idx), abs(scale) * (np.abs(gw) + mean_abs) / P)
    g = np.zeros(E)
    if grad_loss is not None:
        C = float(np.sum(counts))
        g = float(grad_loss) * loss_coef * E * K / C ** 2 * np.asarray(counts, np.float64) if C else g
    if sigmoid:
        z = p.sum(1, keepdims=True) + 1e-20
        with np.errstate(over="ignore"):
            q = 1.0 / (1.0 + np.exp(clean(logits)))
        out = (d + (g - (g * h).sum(1, keepdims=True)) / z) * p * q
        A = (A + (np.abs(g) + (np.abs(g) * h).sum(1, keepdims=True)) / z) * p * q
    else:
        d = d + g
        A = A + np.abs(g)
        out = p * (d - (d * p).sum(1, keepdims=True))
        A = p * (A + (A * p).sum(1, keepdims=True))
    live = r["live"][:, None]
    return np.where(live, out, 0.0), np.where(live, A, 0.0)


def router_units(logits):
    """How many half steps of fp32 (U) a probability may be off: the rounding of l - max
    (|l - max| half steps of the exponent's argument), expf (2 steps = 4 U), a warp's sum
    (up to 32 + 5 additions), the reciprocal and products (8)."""
    l = clean(logits)
    fin = l[np.isfinite(l) & (np.abs(l) < 1e30)]
    span = float(fin.max() - fin.min()) if fin.size else 0.0
    return span + 4 + 37 + 8


E4M3 = np.array([(-1.0 if c >> 7 else 1.0) * (((c & 7) / 8.0) * 2.0 ** -6 if (c >> 3 & 15) == 0
                                             else (1 + (c & 7) / 8.0) * 2.0 ** ((c >> 3 & 15) - 7)) for c in range(256)])


def decode8(q, sf):
    """Values of a row-wise pair (numpy uint8), float64."""
    return E4M3[q] * np.repeat(2.0 ** (sf.astype(np.float64) - 127), 128, axis=1)


def encode8(x):
    """The row-wise pair of exact values x (float64 [rows, cols]): least e with amax <= 448 * 2^e
    (0 for a zero tile, at least -127), nearest code, ties to the even one."""
    rows, cols = x.shape
    t = x.reshape(rows, cols // 128, 128)
    amax = np.abs(t).max(2)
    m, p = np.frexp(amax)
    e = np.where(amax == 0, 0, np.maximum(p - 9 + (m > 0.875), -127))
    v = np.abs(t) / 2.0 ** e[..., None].astype(np.float64)
    grid = E4M3[:127]
    hi = np.clip(np.searchsorted(grid, v), 1, 126)
    lo = hi - 1
    a, b = v - grid[lo], grid[hi] - v
    code = np.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)
    code = code + 128 * np.signbit(t)
    return code.astype(np.uint8).reshape(rows, cols), (e + 127).astype(np.uint8)


def swiglu_bwd(g, u, dy, w):
    """(dgate, dup, y, dw) in float64 and, for each, a bound of the fp32 kernel's error.

    The kernel's exp(-g) is off by 1.5 |g| + 4 half steps (the argument's rounding, the
    hardware's exponential), s = 1 / (1 + exp(-g)) by 4 more; 1 - s adds an absolute half
    step, so the slope s (1 + g (1 - s)) is off by that count times s (1 + |g|).  Below
    2^-126 the hardware flushes to zero."""
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
        q = 1.0 / (1.0 + np.exp(g))
    w = np.ones((g.shape[0], 1)) if w is None else np.asarray(w, np.float64)[:, None]
    act, slope = g * s, s * (1.0 + g * q)
    n = 2 * (1.5 * np.abs(g) + 16) * U
    tiny = 2.0 ** -125
    n = np.minimum(n, 1.0)
    mag = s * (1.0 + np.abs(g))
    e_slope, e_act = mag * n + tiny * (1 + np.abs(g)), np.abs(act) * n + tiny * np.abs(g)
    dw_terms = dy * act * u
    cols = g.shape[1]
    return dict(dg=w * dy * u * slope, du=w * dy * act, y=w * act * u, dw=dw_terms.sum(1),
                e_dg=np.abs(w * dy * u) * e_slope, e_du=np.abs(w * dy) * e_act, e_y=np.abs(w * u) * e_act,
                # the terms' errors, and the additions: 16 * ceil(cols / 4096) in a lane, 3, at most 32
                e_dw=(np.abs(dy * u) * e_act).sum(1) + np.abs(dw_terms).sum(1) * (16 * -(-cols // 4096) + 40) * U)


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def encode4(x):
    """(codes u8 [rows, cols/2], scale bytes u8 [rows, cols/32] row-major) of exact values x."""
    rows, cols = x.shape
    t = np.asarray(x, np.float64).reshape(rows, cols // 32, 32)
    amax = np.abs(t).max(2)
    m, p = np.frexp(amax)
    e = np.where(amax == 0, 0, np.maximum(p - 3 + (m > 0.75), -127))
    v = np.abs(t) / 2.0 ** e[..., None].astype(np.float64)
    grid = E2M1[:8]
    hi = np.clip(np.searchsorted(grid, v), 1, 7)
    lo = hi - 1
    a, b = v - grid[lo], grid[hi] - v
    code = np.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi) + 8 * np.signbit(t)
    code = code.astype(np.uint8).reshape(rows, cols // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).astype(np.uint8)


def decode4(q, sf):
    rows, half = q.shape
    v = np.stack([E2M1[q & 15], E2M1[q >> 4]], 2).reshape(rows, 2 * half)
    return v * np.repeat(2.0 ** (sf.astype(np.float64) - 127), 32, axis=1)


def tile_scales(sf, fill=127):
    """Row-major scale bytes -> the products' order, one byte at a time by its definition."""
    rows, c = sf.shape
    out = np.full(((rows + 127) // 128) * (c // 4) * 512, fill, np.uint8)
    r, k = np.meshgrid(np.arange(rows), np.arange(c), indexing="ij")
    out[((r // 128) * (c // 4) + k // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + k % 4] = sf
    return out


def matmul_bound(a, b):
    """Error bound of an fp32 tensor-core product rounded to BF16: each MMA of 64 elements
    adds to the accumulator with at most 2^-22 of the magnitudes summed so far, then half a
    BF16 step."""
    k = a.shape[1]
    want = a @ b.T
    return want, (k / 64 + 1) * 2.0 ** -22 * (np.abs(a) @ np.abs(b).T) + np.abs(want) * U_BF16 * 1.01 + 1e-37
