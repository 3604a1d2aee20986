"""Python binding of the operators on either side of the FP8 path of an MoE layer: the
router (top-k, weights, balance loss) and its gradient, the SwiGLU with its 8-bit
checkpoints and its backward pass, and the MXFP4 quantization and products.

As in the package's other calls, the functions named ``fp8q_*`` mirror the C entry points
argument for argument and the lower-case helpers allocate their outputs.  Both check every
tensor (device, type, contiguity, size) before the library sees its address.
"""
from __future__ import annotations

from . import _check, _stream, fp8q_permute_workspace_bytes, lib, permute_max_rows

__all__ = [
    "ROUTER_SIGMOID", "ROUTER_RENORM", "ROUTER_BF16", "fp8q_router_workspace_bytes", "fp8q_router_topk",
    "fp8q_router_topk_bwd", "fp8q_permute_row_weights", "router_topk", "router_topk_bwd", "permute_row_weights",
    "fp8q_swiglu_quant_stash", "fp8q_swiglu_bwd", "fp8q_swiglu_bwd_quant", "swiglu_quant_stash", "swiglu_bwd",
    "swiglu_bwd_quant",
    "fp8q_mxfp4_sf_bytes", "fp8q_quantize_rowwise_mxfp4", "fp8q_permute_pad_mxfp4", "fp8q_matmul_mxfp4",
    "mxfp4_tile_scales", "quantize_rowwise_mxfp4", "permute_pad_mxfp4", "matmul_mxfp4",
]

ROUTER_SIGMOID = 0x1  # FP8Q_ROUTER_SIGMOID
ROUTER_RENORM = 0x2   # FP8Q_ROUTER_RENORM
ROUTER_BF16 = 0x4     # FP8Q_ROUTER_BF16


def _in(t, name: str, dtypes, numel: int):
    """Address of a tensor of at least `numel` elements of one of the types, contiguous and
    on the current CUDA device; None -> NULL."""
    import torch
    if t is None:
        return None
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: libfp8q takes tensors on the current CUDA device, got one on {t.device}")
    if t.dtype not in (dtypes if isinstance(dtypes, tuple) else (dtypes,)):
        raise ValueError(f"{name}: unexpected type {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: libfp8q takes contiguous tensors")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, {numel} needed")
    return t.data_ptr() if t.numel() else None


def _shape(t, name: str, shape) -> None:
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _scratch(nbytes: int, like, stream):
    """Workspace of one call, kept from reuse until the work on `stream` is done."""
    import torch
    ws = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=like.device)
    if stream is not None and not torch.cuda.is_current_stream_capturing():
        s = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream
        ws.record_stream(s)
    return ws


# ---------------------------------------------------------------- router
def fp8q_router_workspace_bytes(tokens: int, num_experts: int) -> int:
    return int(lib().fp8q_router_workspace_bytes(tokens, num_experts))


def _logits_type(flags: int):
    import torch
    return torch.bfloat16 if flags & ROUTER_BF16 else torch.float32


def fp8q_router_topk(logits, tokens: int, num_experts: int, flags: int, bias, token_mask, topk: int, scale: float,
                     loss_coef: float, topk_idx, weights, counts, prob_sums, loss, workspace, workspace_bytes: int,
                     stream=None) -> None:
    import torch
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    _check(lib().fp8q_router_topk(
        _in(logits, "logits", _logits_type(flags), tokens * num_experts), tokens, num_experts, flags,
        _in(bias, "bias", f32, num_experts), _in(token_mask, "token_mask", (u8, torch.bool), tokens), topk, scale,
        loss_coef, _in(topk_idx, "topk_idx", i32, tokens * topk), _in(weights, "weights", f32, tokens * topk),
        _in(counts, "counts", i32, num_experts), _in(prob_sums, "prob_sums", f32, num_experts),
        _in(loss, "loss", f32, 1), _in(workspace, "workspace", u8, workspace_bytes), workspace_bytes,
        _stream(stream)), "fp8q_router_topk")


def fp8q_router_topk_bwd(logits, tokens: int, num_experts: int, flags: int, token_mask, topk: int, scale: float,
                         topk_idx, grad_weights, row_id_map, grad_rows: int, counts, loss_coef: float, grad_loss,
                         grad_logits, stream=None) -> None:
    import torch
    f32, i32 = torch.float32, torch.int32
    dt = _logits_type(flags)
    _check(lib().fp8q_router_topk_bwd(
        _in(logits, "logits", dt, tokens * num_experts), tokens, num_experts, flags,
        _in(token_mask, "token_mask", (torch.uint8, torch.bool), tokens), topk, scale,
        _in(topk_idx, "topk_idx", i32, tokens * topk),
        _in(grad_weights, "grad_weights", f32, tokens * topk if row_id_map is None else grad_rows),
        _in(row_id_map, "row_id_map", i32, tokens * topk), grad_rows, _in(counts, "counts", i32, num_experts),
        loss_coef, _in(grad_loss, "grad_loss", f32, 1), _in(grad_logits, "grad_logits", dt, tokens * num_experts),
        _stream(stream)), "fp8q_router_topk_bwd")


def fp8q_permute_row_weights(weights, row_id_map, pairs: int, rows: int, row_weights, stream=None) -> None:
    import torch
    _check(lib().fp8q_permute_row_weights(
        _in(weights, "weights", torch.float32, pairs), _in(row_id_map, "row_id_map", torch.int32, pairs), pairs, rows,
        _in(row_weights, "row_weights", torch.float32, rows), _stream(stream)), "fp8q_permute_row_weights")


def _router_flags(logits, sigmoid: bool, renormalize: bool) -> int:
    import torch
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"logits: fp32 or BF16, got {logits.dtype}")
    return ((ROUTER_SIGMOID if sigmoid else 0) | (ROUTER_RENORM if renormalize else 0)
            | (ROUTER_BF16 if logits.dtype == torch.bfloat16 else 0))


def router_topk(logits, topk: int, *, sigmoid: bool = False, renormalize: bool = True, bias=None, token_mask=None,
                scale: float = 1.0, balance: bool = True, loss_coef: float = 1.0, stream=None):
    """logits [tokens, experts] (fp32 or BF16) -> (topk_idx int32 [tokens, topk], weights fp32
    [tokens, topk], counts int32 [experts], prob_sums fp32 [experts], loss fp32 [1]); the
    last three are None without `balance` (serving)."""
    import torch
    tokens, experts = logits.shape
    _shape(bias, "bias", (experts,))
    _shape(token_mask, "token_mask", (tokens,))
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device=logits.device)  # noqa: E731
    idx, weights = new((tokens, topk), torch.int32), new((tokens, topk), torch.float32)
    counts = sums = loss = ws = None
    if balance:
        counts, sums, loss = new((experts,), torch.int32), new((experts,), torch.float32), new((1,), torch.float32)
        ws = _scratch(fp8q_router_workspace_bytes(tokens, experts), logits, stream)
    fp8q_router_topk(logits, tokens, experts, _router_flags(logits, sigmoid, renormalize), bias, token_mask, topk,
                     scale, loss_coef, idx, weights, counts, sums, loss, ws, ws.numel() if balance else 0, stream)
    return idx, weights, counts, sums, loss


def router_topk_bwd(logits, topk_idx, grad_weights=None, *, row_id_map=None, counts=None, grad_loss=None,
                    sigmoid: bool = False, renormalize: bool = True, token_mask=None, scale: float = 1.0,
                    loss_coef: float = 1.0, stream=None):
    """Gradient of the logits.  grad_weights: fp32 [tokens, topk], or with row_id_map fp32
    [rows] in a permute's row order; grad_loss: fp32 [1] on the device, with the counts of
    the forward call.  The other arguments as in router_topk."""
    import torch
    tokens, experts = logits.shape
    topk = topk_idx.shape[1]
    _shape(topk_idx, "topk_idx", (tokens, topk))
    _shape(token_mask, "token_mask", (tokens,))
    rows = 0
    if row_id_map is not None:
        if row_id_map.numel() != tokens * topk or grad_weights is None:
            raise ValueError("row_id_map: one entry per (token, slot) pair, with grad_weights in row order")
        rows = grad_weights.numel()
    else:
        _shape(grad_weights, "grad_weights", (tokens, topk))
    grad = torch.empty_like(logits)
    fp8q_router_topk_bwd(logits, tokens, experts, _router_flags(logits, sigmoid, renormalize), token_mask, topk, scale,
                         topk_idx, grad_weights, row_id_map, rows, counts, loss_coef, grad_loss, grad, stream)
    return grad


def permute_row_weights(weights, row_id_map, rows: int, stream=None):
    """Routing weights [tokens, topk] -> fp32 [rows] in a permute's row order, 0 elsewhere."""
    import torch
    if weights.numel() != row_id_map.numel():
        raise ValueError("weights and row_id_map: one entry per (token, slot) pair each")
    out = torch.empty((rows,), dtype=torch.float32, device=weights.device)
    fp8q_permute_row_weights(weights, row_id_map, row_id_map.numel(), rows, out, stream)
    return out


# ---------------------------------------------------------------- 8-bit SwiGLU checkpoints
def fp8q_swiglu_quant_stash(gate, up, row_weights, rows: int, cols: int, q, sf, qt, sft, gq, gsf, uq, usf,
                            stream=None) -> None:
    import torch
    bf16, u8, n, t = torch.bfloat16, torch.uint8, rows * cols, rows * (cols // 128)
    _check(lib().fp8q_swiglu_quant_stash(
        _in(gate, "gate", bf16, n), _in(up, "up", bf16, n), _in(row_weights, "row_weights", torch.float32, rows), rows,
        cols, _in(q, "q", u8, n), _in(sf, "sf", u8, t), _in(qt, "qt", u8, n), _in(sft, "sft", u8, t),
        _in(gq, "gq", u8, n), _in(gsf, "gsf", u8, t), _in(uq, "uq", u8, n), _in(usf, "usf", u8, t), _stream(stream)),
        "fp8q_swiglu_quant_stash")


def _bwd_in(gq, gsf, uq, usf, row_weights, dy, rows, cols):
    import torch
    u8, n, t = torch.uint8, rows * cols, rows * (cols // 128)
    return (_in(gq, "gq", u8, n), _in(gsf, "gsf", u8, t), _in(uq, "uq", u8, n), _in(usf, "usf", u8, t),
            _in(row_weights, "row_weights", torch.float32, rows), _in(dy, "dy", torch.bfloat16, n))


def fp8q_swiglu_bwd(gq, gsf, uq, usf, row_weights, dy, rows: int, cols: int, dgate, dup, drow_weights,
                    stream=None) -> None:
    import torch
    bf16, n = torch.bfloat16, rows * cols
    _check(lib().fp8q_swiglu_bwd(
        *_bwd_in(gq, gsf, uq, usf, row_weights, dy, rows, cols), rows, cols, _in(dgate, "dgate", bf16, n),
        _in(dup, "dup", bf16, n), _in(drow_weights, "drow_weights", torch.float32, rows), _stream(stream)),
        "fp8q_swiglu_bwd")


def fp8q_swiglu_bwd_quant(gq, gsf, uq, usf, row_weights, dy, rows: int, cols: int, dgq, dgsf, duq, dusf, yq, ysf,
                          drow_weights, stream=None) -> None:
    import torch
    u8, n, t = torch.uint8, rows * cols, rows * (cols // 128)
    _check(lib().fp8q_swiglu_bwd_quant(
        *_bwd_in(gq, gsf, uq, usf, row_weights, dy, rows, cols), rows, cols, _in(dgq, "dgq", u8, n),
        _in(dgsf, "dgsf", u8, t), _in(duq, "duq", u8, n), _in(dusf, "dusf", u8, t), _in(yq, "yq", u8, n),
        _in(ysf, "ysf", u8, t), _in(drow_weights, "drow_weights", torch.float32, rows), _stream(stream)),
        "fp8q_swiglu_bwd_quant")


def _pair(shape, like):
    """Codes [rows, cols] and scales [rows, cols/128] of a row-wise pair."""
    import torch
    rows, cols = shape
    return (torch.empty((rows, cols), dtype=torch.uint8, device=like.device),
            torch.empty((rows, cols // 128), dtype=torch.uint8, device=like.device))


def swiglu_quant_stash(gate, up, row_weights=None, stream=None):
    """y = silu(gate) * up (* row_weights) as a row-wise pair, and gate and up as row-wise
    pairs for swiglu_bwd: (q, sf, gq, gsf, uq, usf)."""
    rows, cols = gate.shape
    _shape(up, "up", (rows, cols))
    _shape(row_weights, "row_weights", (rows,))
    q, sf = _pair((rows, cols), gate)
    gq, gsf = _pair((rows, cols), gate)
    uq, usf = _pair((rows, cols), gate)
    fp8q_swiglu_quant_stash(gate, up, row_weights, rows, cols, q, sf, None, None, gq, gsf, uq, usf, stream)
    return q, sf, gq, gsf, uq, usf


def _bwd_shapes(gq, gsf, uq, usf, dy, row_weights):
    rows, cols = gq.shape
    for t, name in ((uq, "uq"), (dy, "dy")):
        _shape(t, name, (rows, cols))
    for t, name in ((gsf, "gsf"), (usf, "usf")):
        _shape(t, name, (rows, cols // 128))
    _shape(row_weights, "row_weights", (rows,))
    return rows, cols


def swiglu_bwd(gq, gsf, uq, usf, dy, row_weights=None, stream=None):
    """Gradients of gate and up (BF16) and of the row weights (fp32, None without them) from
    the 8-bit checkpoints and dy, the BF16 gradient of the forward's y."""
    import torch
    rows, cols = _bwd_shapes(gq, gsf, uq, usf, dy, row_weights)
    dg, du = torch.empty_like(dy), torch.empty_like(dy)
    dw = None if row_weights is None else torch.empty_like(row_weights)
    fp8q_swiglu_bwd(gq, gsf, uq, usf, row_weights, dy, rows, cols, dg, du, dw, stream)
    return dg, du, dw


def swiglu_bwd_quant(gq, gsf, uq, usf, dy, row_weights=None, recompute: bool = True, stream=None):
    """The same gradients as row-wise E4M3 pairs, with y recomputed from the checkpoints:
    (dgq, dgsf, duq, dusf, yq, ysf, drow_weights); yq, ysf are None without `recompute`."""
    import torch
    rows, cols = _bwd_shapes(gq, gsf, uq, usf, dy, row_weights)
    dgq, dgsf = _pair((rows, cols), gq)
    duq, dusf = _pair((rows, cols), gq)
    yq, ysf = _pair((rows, cols), gq) if recompute else (None, None)
    dw = None if row_weights is None else torch.empty_like(row_weights)
    fp8q_swiglu_bwd_quant(gq, gsf, uq, usf, row_weights, dy, rows, cols, dgq, dgsf, duq, dusf, yq, ysf, dw, stream)
    return dgq, dgsf, duq, dusf, yq, ysf, dw


# ---------------------------------------------------------------- MXFP4
def fp8q_mxfp4_sf_bytes(rows: int, k: int) -> int:
    return int(lib().fp8q_mxfp4_sf_bytes(rows, k))


def fp8q_quantize_rowwise_mxfp4(x, rows: int, cols: int, q, sf, stream=None) -> None:
    import torch
    u8 = torch.uint8
    _check(lib().fp8q_quantize_rowwise_mxfp4(
        _in(x, "x", torch.bfloat16, rows * cols), rows, cols, _in(q, "q", u8, rows * (cols // 2)),
        _in(sf, "sf", u8, fp8q_mxfp4_sf_bytes(rows, cols)), _stream(stream)), "fp8q_quantize_rowwise_mxfp4")


def fp8q_permute_pad_mxfp4(x, tokens: int, hidden: int, topk_idx, topk: int, num_experts: int, align: int, q, sf,
                           max_out_rows: int, expert_offsets, row_id_map, workspace, workspace_bytes: int,
                           stream=None) -> None:
    import torch
    u8, i32 = torch.uint8, torch.int32
    _check(lib().fp8q_permute_pad_mxfp4(
        _in(x, "x", torch.bfloat16, tokens * hidden), tokens, hidden, _in(topk_idx, "topk_idx", i32, tokens * topk),
        topk, num_experts, align, _in(q, "q", u8, max_out_rows * (hidden // 2)),
        _in(sf, "sf", u8, fp8q_mxfp4_sf_bytes(max_out_rows, hidden)), max_out_rows,
        _in(expert_offsets, "expert_offsets", i32, num_experts + 1), _in(row_id_map, "row_id_map", i32, tokens * topk),
        _in(workspace, "workspace", u8, workspace_bytes), workspace_bytes, _stream(stream)), "fp8q_permute_pad_mxfp4")


def fp8q_matmul_mxfp4(aq, asf, m: int, bq, bsf, n: int, k: int, group_offsets, num_groups: int, out,
                      stream=None) -> None:
    import torch
    u8, b_rows = torch.uint8, n * num_groups
    _check(lib().fp8q_matmul_mxfp4(
        _in(aq, "aq", u8, m * (k // 2)), _in(asf, "asf", u8, fp8q_mxfp4_sf_bytes(m, k)), m,
        _in(bq, "bq", u8, b_rows * (k // 2)), _in(bsf, "bsf", u8, fp8q_mxfp4_sf_bytes(b_rows, k)), n, k,
        _in(group_offsets, "group_offsets", torch.int32, num_groups + 1), num_groups,
        _in(out, "out", torch.bfloat16, m * n), _stream(stream)), "fp8q_matmul_mxfp4")


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


def quantize_rowwise_mxfp4(x, stream=None):
    """x: bf16 [rows, cols] -> (q u8 [rows, cols/2], sf u8 flat, in the products' order)."""
    import torch
    rows, cols = x.shape
    q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
    sf = torch.empty((fp8q_mxfp4_sf_bytes(rows, cols),), dtype=torch.uint8, device=x.device)
    fp8q_quantize_rowwise_mxfp4(x, rows, cols, q, sf, stream)
    return q, sf


def permute_pad_mxfp4(x, topk_idx, num_experts: int, align: int, max_out_rows: int | None = None, stream=None):
    """permute_pad_quant with 4-bit rows: (q u8 [max_out_rows, hidden/2], sf, expert_offsets
    [E+1], row_id_map [T*K])."""
    import torch
    tokens, hidden = x.shape
    topk = topk_idx.shape[1]
    _shape(topk_idx, "topk_idx", (tokens, topk))
    if max_out_rows is None:
        max_out_rows = permute_max_rows(tokens, topk, num_experts, align)
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device=x.device)  # noqa: E731
    q = new((max_out_rows, hidden // 2), torch.uint8)
    sf = new((fp8q_mxfp4_sf_bytes(max_out_rows, hidden),), torch.uint8)
    off, rmap = new((num_experts + 1,), torch.int32), new((tokens * topk,), torch.int32)
    ws = _scratch(fp8q_permute_workspace_bytes(tokens, topk, num_experts), x, stream)
    fp8q_permute_pad_mxfp4(x, tokens, hidden, topk_idx, topk, num_experts, align, q, sf, max_out_rows, off, rmap, ws,
                           ws.numel(), stream)
    return q, sf, off, rmap


def matmul_mxfp4(aq, asf, bq, bsf, group_offsets=None, out=None, stream=None):
    """BF16 [m, n] = A [m, k] times B [n, k] transposed, both MXFP4 (codes [rows, k/2], scales in
    the products' order).  With group_offsets (device int32 [G+1], as the permutes write them
    with align 128) bq is [G*n, k/2]: rows of group g are multiplied by its n rows; rows of
    out past the last group are not written (pass `out` to say what they hold)."""
    import torch
    m, k = aq.shape[0], 2 * aq.shape[1]
    groups = 1 if group_offsets is None else group_offsets.numel() - 1
    if bq.shape[1] * 2 != k or groups < 1 or bq.shape[0] % groups:
        raise ValueError(f"codes {tuple(aq.shape)} and {tuple(bq.shape)} do not fit ({groups} groups)")
    n = bq.shape[0] // groups
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=aq.device)
    _shape(out, "out", (m, n))
    fp8q_matmul_mxfp4(aq, asf, m, bq, bsf, n, k, group_offsets, groups, out, stream)
    return out
