"""Python binding of the operators on either side of the FP8 path of an MoE layer: the
router (top-k, weights, balance loss) and its gradient, the SwiGLU with its 8-bit
checkpoints and its backward pass, and the MXFP4 quantization and products.

As in the package's other calls, the functions named ``fp8q_*`` mirror the C entry points
argument for argument and the lower-case helpers allocate their outputs.  Both check every
tensor that the caller gives (device, type, contiguity, size) before the library sees its
address.  A helper given a ``stream`` allocates and launches on that stream.
"""
from __future__ import annotations

import functools

from . import _check, lib, permute_max_rows

__all__ = [
    "ROUTER_SIGMOID", "ROUTER_RENORM", "ROUTER_BF16", "fp8q_router_workspace_bytes", "fp8q_router_topk",
    "fp8q_router_topk_bwd", "fp8q_permute_row_weights", "router_topk", "router_topk_bwd", "permute_row_weights",
    "fp8q_swiglu_quant_stash", "fp8q_swiglu_bwd", "fp8q_swiglu_bwd_quant", "swiglu_quant_stash", "swiglu_bwd",
    "swiglu_bwd_quant", "fp8q_mxfp4_sf_bytes", "fp8q_quantize_rowwise_mxfp4", "fp8q_permute_pad_mxfp4",
    "fp8q_matmul_mxfp4", "mxfp4_tile_scales", "quantize_rowwise_mxfp4", "permute_pad_mxfp4", "matmul_mxfp4",
]

ROUTER_SIGMOID = 0x1  # FP8Q_ROUTER_SIGMOID
ROUTER_RENORM = 0x2   # FP8Q_ROUTER_RENORM
ROUTER_BF16 = 0x4     # FP8Q_ROUTER_BF16


# ---------------------------------------------------------------- marshalling
# A call costs a few microseconds on the host, which is what bounds the small sizes: one
# query of the device and of its stream a call, plain integers for addresses.
def _device() -> int:
    import torch
    return torch._C._cuda_getDevice()


def _raw_stream(stream, dev: int) -> int:
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _in(t, name: str, dtype, numel: int, dev: int):
    """Address of a tensor of at least `numel` elements of the type, contiguous and on the
    current CUDA device `dev`; None -> NULL."""
    if t is None:
        return None
    if t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous() or t.numel() < numel:
        _refuse(t, name, dtype, numel, dev)
    return t.data_ptr()


def _refuse(t, name, dtype, numel, dev):
    if t.get_device() != dev:
        raise ValueError(f"{name}: libfp8q takes tensors on the current CUDA device, got one on {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: libfp8q takes contiguous tensors")
    raise ValueError(f"{name}: {t.numel()} elements, {numel} needed")


def _mask(t, tokens: int, dev: int):
    """Address of a token mask, uint8 or bool."""
    import torch
    return _in(t, "token_mask", torch.bool if t is not None and t.dtype is torch.bool else torch.uint8, tokens, dev)


def _shape(t, name: str, shape) -> None:
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _helper(fn):
    """Adds the keyword `stream`: the helper then runs, allocations included, with that
    stream current (memory of another stream's pool could still be in use there)."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        import torch
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


# ---------------------------------------------------------------- router
def fp8q_router_workspace_bytes(tokens: int, num_experts: int) -> int:
    return lib().fp8q_router_workspace_bytes(tokens, num_experts)


def _logits_type(flags: int):
    import torch
    return torch.bfloat16 if flags & ROUTER_BF16 else torch.float32


def fp8q_router_topk(logits, tokens: int, num_experts: int, flags: int, bias, token_mask, topk: int, scale: float,
                     loss_coef: float, topk_idx, weights, counts, prob_sums, loss, workspace, workspace_bytes: int,
                     stream=None) -> None:
    import torch
    f32, i32, u8, dev = torch.float32, torch.int32, torch.uint8, _device()
    _check(lib().fp8q_router_topk(
        _in(logits, "logits", _logits_type(flags), tokens * num_experts, dev), tokens, num_experts, flags,
        _in(bias, "bias", f32, num_experts, dev), _mask(token_mask, tokens, dev), topk, scale, loss_coef,
        _in(topk_idx, "topk_idx", i32, tokens * topk, dev), _in(weights, "weights", f32, tokens * topk, dev),
        _in(counts, "counts", i32, num_experts, dev), _in(prob_sums, "prob_sums", f32, num_experts, dev),
        _in(loss, "loss", f32, 1, dev), _in(workspace, "workspace", u8, workspace_bytes, dev), workspace_bytes,
        _raw_stream(stream, dev)), "fp8q_router_topk")


def fp8q_router_topk_bwd(logits, tokens: int, num_experts: int, flags: int, token_mask, topk: int, scale: float,
                         topk_idx, grad_weights, row_id_map, grad_rows: int, counts, loss_coef: float, grad_loss,
                         grad_logits, stream=None) -> None:
    import torch
    f32, i32, dt, dev = torch.float32, torch.int32, _logits_type(flags), _device()
    _check(lib().fp8q_router_topk_bwd(
        _in(logits, "logits", dt, tokens * num_experts, dev), tokens, num_experts, flags,
        _mask(token_mask, tokens, dev), topk, scale, _in(topk_idx, "topk_idx", i32, tokens * topk, dev),
        _in(grad_weights, "grad_weights", f32, tokens * topk if row_id_map is None else grad_rows, dev),
        _in(row_id_map, "row_id_map", i32, tokens * topk, dev), grad_rows,
        _in(counts, "counts", i32, num_experts, dev), loss_coef, _in(grad_loss, "grad_loss", f32, 1, dev),
        _in(grad_logits, "grad_logits", dt, tokens * num_experts, dev), _raw_stream(stream, dev)),
        "fp8q_router_topk_bwd")


def fp8q_permute_row_weights(weights, row_id_map, pairs: int, rows: int, row_weights, stream=None) -> None:
    import torch
    f32, dev = torch.float32, _device()
    _check(lib().fp8q_permute_row_weights(
        _in(weights, "weights", f32, pairs, dev), _in(row_id_map, "row_id_map", torch.int32, pairs, dev), pairs, rows,
        _in(row_weights, "row_weights", f32, rows, dev), _raw_stream(stream, dev)), "fp8q_permute_row_weights")


def _router_flags(logits, sigmoid: bool, renormalize: bool):
    """(flags, type) of a router call."""
    import torch
    dt = logits.dtype
    if dt is torch.float32:
        flags = 0
    elif dt is torch.bfloat16:
        flags = ROUTER_BF16
    else:
        raise ValueError(f"logits: fp32 or BF16, got {dt}")
    return flags | (ROUTER_SIGMOID if sigmoid else 0) | (ROUTER_RENORM if renormalize else 0), dt


@_helper
def router_topk(logits, topk: int, *, sigmoid: bool = False, renormalize: bool = True, bias=None, token_mask=None,
                scale: float = 1.0, balance: bool = True, loss_coef: float = 1.0):
    """logits [tokens, experts] (fp32 or BF16) -> (topk_idx int32 [tokens, topk], weights fp32
    [tokens, topk], counts int32 [experts], prob_sums fp32 [experts], loss fp32 [1]); the
    last three are None without `balance` (serving)."""
    import torch
    tokens, experts = logits.shape
    flags, dt = _router_flags(logits, sigmoid, renormalize)
    f32, i32, dev = torch.float32, torch.int32, _device()
    if bias is not None:
        _shape(bias, "bias", (experts,))
    if token_mask is not None:
        _shape(token_mask, "token_mask", (tokens,))
    lp = _in(logits, "logits", dt, 0, dev)
    bp, mp = _in(bias, "bias", f32, experts, dev), _mask(token_mask, tokens, dev)
    device = logits.device
    idx = torch.empty(tokens, max(topk, 0), dtype=i32, device=device)
    weights = torch.empty_like(idx, dtype=f32)
    if not balance:
        _check(lib().fp8q_router_topk(lp, tokens, experts, flags, bp, mp, topk, scale, loss_coef, idx.data_ptr(),
                                      weights.data_ptr(), None, None, None, None, 0, _raw_stream(None, dev)),
               "fp8q_router_topk")
        return idx, weights, None, None, None
    counts = torch.empty(experts, dtype=i32, device=device)
    sums = torch.empty_like(counts, dtype=f32)
    loss = torch.empty(1, dtype=f32, device=device)
    need = fp8q_router_workspace_bytes(tokens, experts)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    _check(lib().fp8q_router_topk(lp, tokens, experts, flags, bp, mp, topk, scale, loss_coef, idx.data_ptr(),
                                  weights.data_ptr(), counts.data_ptr(), sums.data_ptr(), loss.data_ptr(),
                                  ws.data_ptr(), need, _raw_stream(None, dev)), "fp8q_router_topk")
    return idx, weights, counts, sums, loss


@_helper
def router_topk_bwd(logits, topk_idx, grad_weights=None, *, row_id_map=None, counts=None, grad_loss=None,
                    sigmoid: bool = False, renormalize: bool = True, token_mask=None, scale: float = 1.0,
                    loss_coef: float = 1.0):
    """Gradient of the logits.  grad_weights: fp32 [tokens, topk], or with row_id_map fp32
    [rows] in a permute's row order; grad_loss: fp32 [1] on the device, with the counts of
    the forward call.  The other arguments as in router_topk."""
    import torch
    tokens, experts = logits.shape
    topk = topk_idx.shape[1]
    flags, dt = _router_flags(logits, sigmoid, renormalize)
    f32, i32, dev = torch.float32, torch.int32, _device()
    _shape(topk_idx, "topk_idx", (tokens, topk))
    if token_mask is not None:
        _shape(token_mask, "token_mask", (tokens,))
    rows = 0
    if row_id_map is not None:
        if row_id_map.numel() != tokens * topk or grad_weights is None:
            raise ValueError("row_id_map: one entry per (token, slot) pair, with grad_weights in row order")
        rows = grad_weights.numel()
    elif grad_weights is not None:
        _shape(grad_weights, "grad_weights", (tokens, topk))
    lp = _in(logits, "logits", dt, 0, dev)
    grad = torch.empty_like(logits)
    _check(lib().fp8q_router_topk_bwd(
        lp, tokens, experts, flags, _mask(token_mask, tokens, dev), topk, scale, _in(topk_idx, "topk_idx", i32, 0, dev),
        _in(grad_weights, "grad_weights", f32, 0, dev), _in(row_id_map, "row_id_map", i32, 0, dev), rows,
        _in(counts, "counts", i32, experts, dev), loss_coef, _in(grad_loss, "grad_loss", f32, 1, dev), grad.data_ptr(),
        _raw_stream(None, dev)), "fp8q_router_topk_bwd")
    return grad


@_helper
def permute_row_weights(weights, row_id_map, rows: int):
    """Routing weights [tokens, topk] -> fp32 [rows] in a permute's row order, 0 elsewhere."""
    import torch
    if weights.numel() != row_id_map.numel():
        raise ValueError("weights and row_id_map: one entry per (token, slot) pair each")
    out = torch.empty(rows, dtype=torch.float32, device=weights.device)
    fp8q_permute_row_weights(weights, row_id_map, row_id_map.numel(), rows, out)
    return out


# ---------------------------------------------------------------- 8-bit SwiGLU checkpoints
def fp8q_swiglu_quant_stash(gate, up, row_weights, rows: int, cols: int, q, sf, gq, gsf, uq, usf,
                            stream=None) -> None:
    import torch
    bf16, u8, dev, n, t = torch.bfloat16, torch.uint8, _device(), rows * cols, rows * (cols // 128)
    _check(lib().fp8q_swiglu_quant_stash(
        _in(gate, "gate", bf16, n, dev), _in(up, "up", bf16, n, dev),
        _in(row_weights, "row_weights", torch.float32, rows, dev), rows, cols, _in(q, "q", u8, n, dev),
        _in(sf, "sf", u8, t, dev), _in(gq, "gq", u8, n, dev),
        _in(gsf, "gsf", u8, t, dev), _in(uq, "uq", u8, n, dev), _in(usf, "usf", u8, t, dev), _raw_stream(stream, dev)),
        "fp8q_swiglu_quant_stash")


def _bwd_in(gq, gsf, uq, usf, row_weights, dy, rows, cols, dev):
    import torch
    u8, n, t = torch.uint8, rows * cols, rows * (cols // 128)
    return (_in(gq, "gq", u8, n, dev), _in(gsf, "gsf", u8, t, dev), _in(uq, "uq", u8, n, dev),
            _in(usf, "usf", u8, t, dev), _in(row_weights, "row_weights", torch.float32, rows, dev),
            _in(dy, "dy", torch.bfloat16, n, dev))


def fp8q_swiglu_bwd(gq, gsf, uq, usf, row_weights, dy, rows: int, cols: int, dgate, dup, drow_weights,
                    stream=None) -> None:
    import torch
    bf16, dev, n = torch.bfloat16, _device(), rows * cols
    _check(lib().fp8q_swiglu_bwd(
        *_bwd_in(gq, gsf, uq, usf, row_weights, dy, rows, cols, dev), rows, cols, _in(dgate, "dgate", bf16, n, dev),
        _in(dup, "dup", bf16, n, dev), _in(drow_weights, "drow_weights", torch.float32, rows, dev),
        _raw_stream(stream, dev)), "fp8q_swiglu_bwd")


def fp8q_swiglu_bwd_quant(gq, gsf, uq, usf, row_weights, dy, rows: int, cols: int, dgq, dgsf, duq, dusf, yq, ysf,
                          drow_weights, stream=None) -> None:
    import torch
    u8, dev, n, t = torch.uint8, _device(), rows * cols, rows * (cols // 128)
    _check(lib().fp8q_swiglu_bwd_quant(
        *_bwd_in(gq, gsf, uq, usf, row_weights, dy, rows, cols, dev), rows, cols, _in(dgq, "dgq", u8, n, dev),
        _in(dgsf, "dgsf", u8, t, dev), _in(duq, "duq", u8, n, dev), _in(dusf, "dusf", u8, t, dev),
        _in(yq, "yq", u8, n, dev), _in(ysf, "ysf", u8, t, dev),
        _in(drow_weights, "drow_weights", torch.float32, rows, dev), _raw_stream(stream, dev)),
        "fp8q_swiglu_bwd_quant")


def _pair(rows: int, cols: int, device):
    """Codes [rows, cols] and scales [rows, cols/128] of a row-wise pair."""
    import torch
    return (torch.empty(rows, cols, dtype=torch.uint8, device=device),
            torch.empty(rows, cols // 128, dtype=torch.uint8, device=device))


@_helper
def swiglu_quant_stash(gate, up, row_weights=None):
    """y = silu(gate) * up (* row_weights) as a row-wise pair, and gate and up as row-wise
    pairs for swiglu_bwd: (q, sf, gq, gsf, uq, usf)."""
    import torch
    rows, cols = gate.shape
    bf16, dev, device = torch.bfloat16, _device(), gate.device
    _shape(up, "up", (rows, cols))
    if row_weights is not None:
        _shape(row_weights, "row_weights", (rows,))
    ins = (_in(gate, "gate", bf16, 0, dev), _in(up, "up", bf16, 0, dev),
           _in(row_weights, "row_weights", torch.float32, 0, dev))
    q, sf = _pair(rows, cols, device)
    gq, gsf, uq, usf = (torch.empty_like(t) for t in (q, sf, q, sf))
    _check(lib().fp8q_swiglu_quant_stash(
        *ins, rows, cols, q.data_ptr(), sf.data_ptr(), gq.data_ptr(), gsf.data_ptr(), uq.data_ptr(),
        usf.data_ptr(), _raw_stream(None, dev)), "fp8q_swiglu_quant_stash")
    return q, sf, gq, gsf, uq, usf


def _bwd_shapes(gq, gsf, uq, usf, dy, row_weights):
    rows, cols = gq.shape
    for t, name, c in ((uq, "uq", cols), (dy, "dy", cols), (gsf, "gsf", cols // 128), (usf, "usf", cols // 128)):
        _shape(t, name, (rows, c))
    if row_weights is not None:
        _shape(row_weights, "row_weights", (rows,))
    return rows, cols


@_helper
def swiglu_bwd(gq, gsf, uq, usf, dy, row_weights=None):
    """Gradients of gate and up (BF16) and of the row weights (fp32, None without them) from
    the 8-bit checkpoints and dy, the BF16 gradient of the forward's y."""
    import torch
    dev = _device()
    rows, cols = _bwd_shapes(gq, gsf, uq, usf, dy, row_weights)
    ins = _bwd_in(gq, gsf, uq, usf, row_weights, dy, rows, cols, dev)
    dg, du = torch.empty_like(dy), torch.empty_like(dy)
    dw = None if row_weights is None else torch.empty_like(row_weights)
    _check(lib().fp8q_swiglu_bwd(*ins, rows, cols, dg.data_ptr(), du.data_ptr(), None if dw is None else dw.data_ptr(),
                                 _raw_stream(None, dev)), "fp8q_swiglu_bwd")
    return dg, du, dw


@_helper
def swiglu_bwd_quant(gq, gsf, uq, usf, dy, row_weights=None, recompute: bool = True):
    """The same gradients as row-wise E4M3 pairs, with y recomputed from the checkpoints:
    (dgq, dgsf, duq, dusf, yq, ysf, drow_weights); yq, ysf are None without `recompute`."""
    import torch
    dev = _device()
    rows, cols = _bwd_shapes(gq, gsf, uq, usf, dy, row_weights)
    ins = _bwd_in(gq, gsf, uq, usf, row_weights, dy, rows, cols, dev)
    dgq, dgsf, duq, dusf = (torch.empty_like(t) for t in (gq, gsf, gq, gsf))
    yq, ysf = (torch.empty_like(gq), torch.empty_like(gsf)) if recompute else (None, None)
    dw = None if row_weights is None else torch.empty_like(row_weights)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _check(lib().fp8q_swiglu_bwd_quant(*ins, rows, cols, dgq.data_ptr(), dgsf.data_ptr(), duq.data_ptr(),
                                       dusf.data_ptr(), ptr(yq), ptr(ysf), ptr(dw), _raw_stream(None, dev)),
           "fp8q_swiglu_bwd_quant")
    return dgq, dgsf, duq, dusf, yq, ysf, dw


# ---------------------------------------------------------------- MXFP4
def fp8q_mxfp4_sf_bytes(rows: int, k: int) -> int:
    return lib().fp8q_mxfp4_sf_bytes(rows, k)


def fp8q_quantize_rowwise_mxfp4(x, rows: int, cols: int, q, sf, stream=None) -> None:
    import torch
    u8, dev = torch.uint8, _device()
    _check(lib().fp8q_quantize_rowwise_mxfp4(
        _in(x, "x", torch.bfloat16, rows * cols, dev), rows, cols, _in(q, "q", u8, rows * (cols // 2), dev),
        _in(sf, "sf", u8, fp8q_mxfp4_sf_bytes(rows, cols), dev), _raw_stream(stream, dev)),
        "fp8q_quantize_rowwise_mxfp4")


def fp8q_permute_pad_mxfp4(x, tokens: int, hidden: int, topk_idx, topk: int, num_experts: int, align: int, q, sf,
                           max_out_rows: int, expert_offsets, row_id_map, workspace, workspace_bytes: int,
                           stream=None) -> None:
    import torch
    u8, i32, dev = torch.uint8, torch.int32, _device()
    _check(lib().fp8q_permute_pad_mxfp4(
        _in(x, "x", torch.bfloat16, tokens * hidden, dev), tokens, hidden,
        _in(topk_idx, "topk_idx", i32, tokens * topk, dev), topk, num_experts, align,
        _in(q, "q", u8, max_out_rows * (hidden // 2), dev),
        _in(sf, "sf", u8, fp8q_mxfp4_sf_bytes(max_out_rows, hidden), dev), max_out_rows,
        _in(expert_offsets, "expert_offsets", i32, num_experts + 1, dev),
        _in(row_id_map, "row_id_map", i32, tokens * topk, dev), _in(workspace, "workspace", u8, workspace_bytes, dev),
        workspace_bytes, _raw_stream(stream, dev)), "fp8q_permute_pad_mxfp4")


def fp8q_matmul_mxfp4(aq, asf, m: int, bq, bsf, n: int, k: int, group_offsets, num_groups: int, out,
                      stream=None) -> None:
    import torch
    u8, dev, b_rows = torch.uint8, _device(), n * num_groups
    _check(lib().fp8q_matmul_mxfp4(
        _in(aq, "aq", u8, m * (k // 2), dev), _in(asf, "asf", u8, fp8q_mxfp4_sf_bytes(m, k), dev), m,
        _in(bq, "bq", u8, b_rows * (k // 2), dev), _in(bsf, "bsf", u8, fp8q_mxfp4_sf_bytes(b_rows, k), dev), n, k,
        _in(group_offsets, "group_offsets", torch.int32, num_groups + 1, dev), num_groups,
        _in(out, "out", torch.bfloat16, m * n, dev), _raw_stream(stream, dev)), "fp8q_matmul_mxfp4")


def mxfp4_tile_scales(sf):
    """Row-major scale bytes u8 [rows, k/32] (k % 128 == 0), as a checkpoint holds them -> the
    tiled order of the products (flat, fp8q_mxfp4_sf_bytes(rows, k) bytes; rows that fill up
    the last 128 get 127).  A layout step for weights, done once when they are loaded."""
    import torch
    rows, c = sf.shape
    if sf.dtype != torch.uint8 or c % 4:
        raise ValueError("scale bytes: uint8 [rows, k/32] with k a multiple of 128")
    blocks = (rows + 127) // 128
    full = torch.full((blocks * 128, c), 127, dtype=torch.uint8, device=sf.device)
    full[:rows] = sf
    return full.view(blocks, 4, 32, c // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


@_helper
def quantize_rowwise_mxfp4(x):
    """x: bf16 [rows, cols] -> (q u8 [rows, cols/2], sf u8 flat, in the products' order)."""
    import torch
    rows, cols = x.shape
    L, u8, dev = lib(), torch.uint8, _device()
    xp = _in(x, "x", torch.bfloat16, 0, dev)
    q = torch.empty(rows, cols // 2, dtype=u8, device=x.device)
    sf = torch.empty(L.fp8q_mxfp4_sf_bytes(rows, cols), dtype=u8, device=x.device)
    _check(L.fp8q_quantize_rowwise_mxfp4(xp, rows, cols, q.data_ptr(), sf.data_ptr(), _raw_stream(None, dev)),
           "fp8q_quantize_rowwise_mxfp4")
    return q, sf


@_helper
def permute_pad_mxfp4(x, topk_idx, num_experts: int, align: int, max_out_rows: int | None = None):
    """permute_pad_quant with 4-bit rows: (q u8 [max_out_rows, hidden/2], sf, expert_offsets
    [E+1], row_id_map [T*K])."""
    import torch
    tokens, hidden = x.shape
    topk = topk_idx.shape[1]
    _shape(topk_idx, "topk_idx", (tokens, topk))
    if max_out_rows is None:
        max_out_rows = permute_max_rows(tokens, topk, num_experts, align)
    L, u8, i32, dev, device = lib(), torch.uint8, torch.int32, _device(), x.device
    xp, ip = _in(x, "x", torch.bfloat16, 0, dev), _in(topk_idx, "topk_idx", i32, 0, dev)
    q = torch.empty(max_out_rows, hidden // 2, dtype=u8, device=device)
    sf = torch.empty(L.fp8q_mxfp4_sf_bytes(max_out_rows, hidden), dtype=u8, device=device)
    off = torch.empty(num_experts + 1, dtype=i32, device=device)
    rmap = torch.empty(tokens * topk, dtype=i32, device=device)
    need = L.fp8q_permute_workspace_bytes(tokens, topk, num_experts)
    ws = torch.empty(max(need, 16), dtype=u8, device=device)
    _check(L.fp8q_permute_pad_mxfp4(xp, tokens, hidden, ip, topk, num_experts, align, q.data_ptr(), sf.data_ptr(),
                                    max_out_rows, off.data_ptr(), rmap.data_ptr(), ws.data_ptr(), need,
                                    _raw_stream(None, dev)), "fp8q_permute_pad_mxfp4")
    return q, sf, off, rmap


@_helper
def matmul_mxfp4(aq, asf, bq, bsf, group_offsets=None, out=None):
    """BF16 [m, n] = A [m, k] times B [n, k] transposed, both MXFP4 (codes [rows, k/2], scales in
    the products' order).  With group_offsets (device int32 [G+1], as the permutes write them
    with align 128) bq is [G*n, k/2]: rows of group g are multiplied by its n rows; rows of
    out past the last group are not written (pass `out` to say what they hold)."""
    import torch
    m, half = aq.shape
    groups = 1 if group_offsets is None else group_offsets.numel() - 1
    if bq.shape[1] != half or groups < 1 or bq.shape[0] % groups:
        raise ValueError(f"codes {tuple(aq.shape)} and {tuple(bq.shape)} do not fit ({groups} groups)")
    n = bq.shape[0] // groups
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=aq.device)
    else:
        _shape(out, "out", (m, n))
    fp8q_matmul_mxfp4(aq, asf, m, bq, bsf, n, 2 * half, group_offsets, groups, out)
    return out
