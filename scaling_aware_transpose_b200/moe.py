"""Python binding of the operators on either side of the FP8 path of an MoE layer: the
router (top-k, weights, balance loss) and its gradient, the SwiGLU with its 8-bit
checkpoints and its backward pass, and the MXFP4 quantization and products.

As in the package's other calls, the functions named ``fp8q_*`` mirror the C entry points
argument for argument and the lower-case helpers allocate their outputs.  Both check every
tensor (device, type, contiguity, size) before the library sees its address.
"""
from __future__ import annotations

from . import _check, _stream, lib

__all__ = [
    "ROUTER_SIGMOID", "ROUTER_RENORM", "ROUTER_BF16", "fp8q_router_workspace_bytes", "fp8q_router_topk",
    "fp8q_router_topk_bwd", "fp8q_permute_row_weights", "router_topk", "router_topk_bwd", "permute_row_weights",
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
