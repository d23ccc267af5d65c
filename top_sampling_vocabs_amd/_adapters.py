"""Low-rank adapters of many requests beside a shared output projection.

The binding of qs_apply_adapters. Like the rest of the binding it only marshals
arguments; it is loaded on first use, because it needs torch at import.
"""

import torch

from ._lib import _check_logits, _status, load
from ._scoring import _addr, _check_out, _check_vec, _code, _enqueue, _refuse_tangents, _wrote


def adapters_workspace_for(logits, rank):
    """A workspace tensor for apply_adapters on these logits. Reuse it across calls on
    one stream, for batches of as many rows or fewer."""
    n = load().qs_adapters_workspace_bytes(int(logits.shape[0]), int(rank))
    return torch.empty(n, dtype=torch.uint8, device=logits.device)


def _check_factor(t, name, shape, index):
    if t.dtype is not torch.bfloat16 or t.dim() != 3 or t.get_device() != index \
            or t.size(2) > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must be a bfloat16 tensor {shape} with unit stride in its last "
                         f"dimension on cuda:{index}")


def _strides(t):
    """(between adapters, between rows); a dimension of one element counts as dense."""
    row = t.stride(1) if t.size(1) > 1 else t.size(2)
    return t.stride(0) if t.size(0) > 1 else 0, row


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
    _check_factor(down, "down", "[count, rank, K]", dev)
    _check_factor(up, "up", "[count, V, rank]", dev)
    count, rank, width = down.shape
    if width != K or up.shape != (count, V, rank):
        raise ValueError(f"down must be [count, rank, {K}] and up [count, {V}, rank], got "
                         f"{list(down.shape)} and {list(up.shape)}")
    _check_vec(index, B, torch.int32, dev, "index")
    if scale is not None:
        _check_vec(scale, count, torch.float32, dev, "scale")
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad
                                       for t in (logits, hidden, down, up, scale)):
        raise ValueError("apply_adapters has no gradient: call it under torch.no_grad() "
                         "or on detached tensors")
    if out is None:
        out = logits
    elif out.shape != logits.shape or out.dtype is not logits.dtype \
            or out.get_device() != dev or out.stride(1) != 1:
        raise ValueError("out must have the logits' shape, dtype and device "
                         "and unit column stride")
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    _check_out(out)
    _refuse_tangents(logits, hidden, down, up, scale, out)
    if workspace is None:
        workspace = adapters_workspace_for(logits, rank)
    status = torch.empty(B, dtype=torch.int32, device=logits.device)
    rc = _enqueue(
        load().qs_apply_adapters, dev,
        logits.data_ptr(), _code(logits, "logits"), B, V, logits.stride(0), hidden.data_ptr(), K,
        hidden.stride(0) if B > 1 else K, down.data_ptr(), *_strides(down), up.data_ptr(),
        *_strides(up), count, rank, index.data_ptr(), _addr(scale), out.data_ptr(), out.stride(0),
        status.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    if rc:
        _status(rc, "qs_apply_adapters")
    _wrote(out)
    return status
