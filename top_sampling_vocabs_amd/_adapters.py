"""Low-rank adapters of many requests beside a shared output projection.

The binding of qs_apply_adapters. Like the rest of the binding it only marshals
arguments; it is loaded on first use, because it needs torch at import.
"""

import functools

import torch

from ._lib import _check_logits, _status, load
from ._scoring import _addr, _check_out, _check_vec, _code, _enqueue, _refuse_tangents, _wrote


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(B, rank):
    # a pure function of its arguments, asked once for each
    return load().qs_adapters_workspace_bytes(B, rank)


def adapters_workspace_for(logits, rank):
    """A workspace tensor for apply_adapters on these logits. Reuse it across calls on
    one stream, for batches of as many rows or fewer."""
    return torch.empty(_workspace_bytes(int(logits.shape[0]), int(rank)), dtype=torch.uint8,
                       device=logits.device)


def _check_factor(t, name, shape, index):
    """t's shape and strides, a dimension of one element counted as dense."""
    if t.dtype is not torch.bfloat16 or t.dim() != 3 or t.get_device() != index:
        raise ValueError(f"{name} must be a bfloat16 tensor {shape} on cuda:{index}")
    (n, rows, columns), (between, row, step) = t.shape, t.stride()
    if step != 1 and columns > 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    return n, rows, columns, between if n > 1 else 0, row if rows > 1 else columns


def apply_adapters(logits, hidden, down, up, index, scale=None, *, out=None, workspace=None):
    """Moves each row's logits by the row's own low-rank adapter of the projection.

    logits [B, V] float32 / bfloat16 (CUDA): head_logits' (or any projection's) of the
    hidden states `hidden` bfloat16 [B, K]; down bfloat16 [count, rank, K] and up
    bfloat16 [count, V, rank], rank a multiple of 8 up to 128; index int32 [B], the
    row's adapter or -1 for none; scale float32 [count] or None (1). To the logits of
    row b is added scale[a] up[a] down[a] hidden[b], a = index[b], in place, or written
    to `out` (the logits' shape and dtype). Returns the row status (int32 [B]):
    ROW_BAD_PARAM for an index that is no adapter, whose row stays as it is. Enqueued
    on the current stream. Inference only: tensors that require a gradient or carry a
    tangent are refused.
    """
    B, V = _check_logits(logits, None)
    dev = logits.get_device()
    if hidden.dtype is not torch.bfloat16 or hidden.dim() != 2 or hidden.size(0) != B \
            or hidden.get_device() != dev or hidden.stride(1) != 1:
        raise ValueError("hidden must be a bfloat16 tensor [B, K] with unit column stride on "
                         f"cuda:{dev}")
    K = hidden.size(1)
    count, rank, width, down_stride, down_row = _check_factor(down, "down", "[count, rank, K]", dev)
    held, rows, ranks, up_stride, up_row = _check_factor(up, "up", "[count, V, rank]", dev)
    if width != K or held != count or rows != V or ranks != rank:
        raise ValueError(f"down must be [count, rank, {K}] and up [count, {V}, rank], got "
                         f"{list(down.shape)} and {list(up.shape)}")
    _check_vec(index, B, torch.int32, dev, "index")
    if scale is not None:
        _check_vec(scale, count, torch.float32, dev, "scale")
    if (logits.requires_grad or hidden.requires_grad or down.requires_grad or up.requires_grad
            or scale is not None and scale.requires_grad) and torch.is_grad_enabled():
        raise ValueError("apply_adapters has no gradient: call it under torch.no_grad() "
                         "or on detached tensors")
    if out is None:
        out = logits
    elif out.shape != logits.shape or out.dtype is not logits.dtype \
            or out.get_device() != dev or out.stride(1) != 1:
        raise ValueError("out must have the logits' shape, dtype and device "
                         "and unit column stride")
    _check_out(out)
    _refuse_tangents(logits, hidden, down, up, scale, out)
    if workspace is None:
        size = _workspace_bytes(B, rank)
        workspace = torch.empty(size, dtype=torch.uint8, device=logits.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    else:
        size = workspace.numel() * workspace.element_size()
    status = torch.empty_like(index)
    rc = _enqueue(
        load().qs_apply_adapters, dev,
        logits.data_ptr(), _code(logits, "logits"), B, V, logits.stride(0), hidden.data_ptr(), K,
        hidden.stride(0) if B > 1 else K, down.data_ptr(), down_stride, down_row, up.data_ptr(),
        up_stride, up_row, count, rank, index.data_ptr(), _addr(scale), out.data_ptr(),
        out.stride(0), status.data_ptr(), workspace.data_ptr(), size)
    if rc:
        _status(rc, "qs_apply_adapters")
    _wrote(out)
    return status
