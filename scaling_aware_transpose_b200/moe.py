"""Python binding of the operators on either side of the FP8 path of an MoE layer: the
router (top-k, weights, balance loss) and its gradient, the SwiGLU with its 8-bit
checkpoints and its backward pass, and the MXFP4 quantization and products.

As in the package's other calls, the functions named ``fp8q_*`` mirror the C entry points
argument for argument and the lower-case helpers allocate their outputs (natively, in
csrc/moe_binding.cpp; a call's small results, such as the scales of its pairs, share one
allocation).  Both check every tensor that the caller gives (device, type,
contiguity, size) before the library sees its address.  A helper given a ``stream``
allocates and launches on that stream.
"""
from __future__ import annotations

from . import _check, lib

__all__ = [
    "ROUTER_SIGMOID", "ROUTER_RENORM", "ROUTER_BF16", "fp8q_router_workspace_bytes", "fp8q_router_topk",
    "fp8q_router_topk_bwd", "fp8q_permute_row_weights", "router_topk", "router_topk_bwd", "permute_row_weights",
    "fp8q_swiglu_quant_stash", "fp8q_swiglu_bwd", "fp8q_swiglu_bwd_quant", "swiglu_quant_stash", "swiglu_bwd",
    "swiglu_bwd_quant", "fp8q_mxfp4_sf_bytes", "fp8q_quantize_rowwise_mxfp4", "fp8q_permute_pad_mxfp4",
    "fp8q_matmul_mxfp4", "fp8q_debug_mxfp4_variant", "mxfp4_tile_scales", "quantize_rowwise_mxfp4", "permute_pad_mxfp4", "matmul_mxfp4",
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


_native = None


def _binding():
    """The native half of the helpers (csrc/moe_binding.cpp); raises if it was not built."""
    global _native
    if _native is None:
        import torch  # its libraries must be loaded first
        lib()
        try:
            from . import _moe_binding
        except ImportError as e:
            raise RuntimeError("_moe_binding.so is missing or does not load; build it with "
                               "`python -m scaling_aware_transpose_b200.build`") from e
        if _moe_binding.torch_version != torch.__version__.split("+")[0]:
            raise RuntimeError(f"_moe_binding.so was built for torch {_moe_binding.torch_version}, this is torch "
                               f"{torch.__version__}; build it with `python -m scaling_aware_transpose_b200.build`")
        _native = _moe_binding
    return _native


def _on(stream, fn, *args):
    """Runs fn, allocations included, with `stream` current (memory of another stream's pool
    could still be in use there)."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return fn(*args)


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


def router_topk(logits, topk: int, *, sigmoid: bool = False, renormalize: bool = True, bias=None, token_mask=None,
                scale: float = 1.0, balance: bool = True, loss_coef: float = 1.0, stream=None):
    """logits [tokens, experts] (fp32 or BF16) -> (topk_idx int32 [tokens, topk], weights fp32
    [tokens, topk], counts int32 [experts], prob_sums fp32 [experts], loss fp32 [1]); the
    last three are None without `balance` (serving)."""
    fn = (_native or _binding()).router_topk
    args = (logits, topk, sigmoid, renormalize, bias, token_mask, scale, balance, loss_coef)
    return fn(*args) if stream is None else _on(stream, fn, *args)


def router_topk_bwd(logits, topk_idx, grad_weights=None, *, row_id_map=None, counts=None, grad_loss=None,
                    sigmoid: bool = False, renormalize: bool = True, token_mask=None, scale: float = 1.0,
                    loss_coef: float = 1.0, stream=None):
    """Gradient of the logits.  grad_weights: fp32 [tokens, topk], or with row_id_map fp32
    [rows] in a permute's row order; grad_loss: fp32 [1] on the device, with the counts of
    the forward call.  The other arguments as in router_topk."""
    fn = (_native or _binding()).router_topk_bwd
    args = (logits, topk_idx, grad_weights, row_id_map, counts, grad_loss, sigmoid, renormalize, token_mask, scale,
            loss_coef)
    return fn(*args) if stream is None else _on(stream, fn, *args)


def permute_row_weights(weights, row_id_map, rows: int, stream=None):
    """Routing weights [tokens, topk] -> fp32 [rows] in a permute's row order, 0 elsewhere."""
    fn = (_native or _binding()).permute_row_weights
    return fn(weights, row_id_map, rows) if stream is None else _on(stream, fn, weights, row_id_map, rows)


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


def swiglu_quant_stash(gate, up, row_weights=None, stream=None):
    """y = silu(gate) * up (* row_weights) as a row-wise pair, and gate and up as row-wise
    pairs for swiglu_bwd: (q, sf, gq, gsf, uq, usf)."""
    fn = (_native or _binding()).swiglu_quant_stash
    return fn(gate, up, row_weights) if stream is None else _on(stream, fn, gate, up, row_weights)


def swiglu_bwd(gq, gsf, uq, usf, dy, row_weights=None, stream=None):
    """Gradients of gate and up (BF16) and of the row weights (fp32, None without them) from
    the 8-bit checkpoints and dy, the BF16 gradient of the forward's y."""
    fn = (_native or _binding()).swiglu_bwd
    args = (gq, gsf, uq, usf, dy, row_weights)
    return fn(*args) if stream is None else _on(stream, fn, *args)


def swiglu_bwd_quant(gq, gsf, uq, usf, dy, row_weights=None, recompute: bool = True, stream=None):
    """The same gradients as row-wise E4M3 pairs, with y recomputed from the checkpoints:
    (dgq, dgsf, duq, dusf, yq, ysf, drow_weights); yq, ysf are None without `recompute`."""
    fn = (_native or _binding()).swiglu_bwd_quant
    args = (gq, gsf, uq, usf, dy, row_weights, recompute)
    return fn(*args) if stream is None else _on(stream, fn, *args)


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


def fp8q_debug_mxfp4_variant(m: int, n: int, k: int, num_groups: int, sms: int):
    """(columns of a tile or 0 for CTA pairs, CTAs that share a tile's k); num_groups 0: dense."""
    import ctypes
    columns, split = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().fp8q_debug_mxfp4_variant(m, n, k, num_groups, sms, ctypes.byref(columns), ctypes.byref(split)),
           "fp8q_debug_mxfp4_variant")
    return columns.value, split.value


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
    fn = (_native or _binding()).quantize_rowwise_mxfp4
    return fn(x) if stream is None else _on(stream, fn, x)


def permute_pad_mxfp4(x, topk_idx, num_experts: int, align: int, max_out_rows: int | None = None, stream=None):
    """permute_pad_quant with 4-bit rows: (q u8 [max_out_rows, hidden/2], sf, expert_offsets
    [E+1], row_id_map [T*K])."""
    fn = (_native or _binding()).permute_pad_mxfp4
    args = (x, topk_idx, num_experts, align, max_out_rows)
    return fn(*args) if stream is None else _on(stream, fn, *args)


def matmul_mxfp4(aq, asf, bq, bsf, group_offsets=None, out=None, stream=None):
    """BF16 [m, n] = A [m, k] times B [n, k] transposed, both MXFP4 (codes [rows, k/2], scales in
    the products' order).  With group_offsets (device int32 [G+1], as the permutes write them
    with align 128) bq is [G*n, k/2]: rows of group g are multiplied by its n rows; rows of
    out past the last group are not written (pass `out` to say what they hold)."""
    fn = (_native or _binding()).matmul_mxfp4
    args = (aq, asf, bq, bsf, group_offsets, out)
    return fn(*args) if stream is None else _on(stream, fn, *args)
