"""Distillation from a teacher's top tokens: the loss and its gradient.

The binding of qs_distill_loss and qs_distill_loss_backward. Like the rest of the
binding it only marshals arguments; it is loaded on first use, because it needs
torch at import.
"""

import functools

import torch

from ._lib import _check_logits, _status, load
from ._scoring import (_addr, _check_out, _check_vec, _code, _enqueue, _padded_rows,
                       _refuse_tangents, _wrote)

STATE = 8  # floats per row that the gradient needs


def _check_inputs(logits, teacher_ids, teacher_values, temperature, bitmask):
    """The forward and the backward call's common inputs: (B, V, K, device index)."""
    B, V = _check_logits(logits, bitmask)
    index = logits.get_device()
    if bitmask is not None and bitmask.get_device() != index:
        raise ValueError(f"bitmask must be on cuda:{index}, got {bitmask.device}")
    if temperature is not None:
        _check_vec(temperature, B, torch.float32, index, "temperature")
    if teacher_ids.dtype is not torch.int32 or teacher_ids.dim() != 2 or teacher_ids.size(0) != B \
            or teacher_ids.get_device() != index or not teacher_ids.is_contiguous():
        raise ValueError(f"teacher_ids must be a contiguous int32 tensor [B, K] on cuda:{index}")
    if teacher_values.dtype is not torch.float32 or teacher_values.shape != teacher_ids.shape \
            or teacher_values.get_device() != index or not teacher_values.is_contiguous():
        raise ValueError("teacher_values must be a contiguous float32 tensor in the shape of "
                         f"teacher_ids on cuda:{index}")
    if torch.is_grad_enabled():
        if teacher_values.requires_grad:
            raise ValueError("the teacher gets no gradient: detach teacher_values")
        if temperature is not None and temperature.requires_grad:
            raise ValueError("temperature gets no gradient: detach it")
    return B, V, teacher_ids.size(1), index


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(B, V, code):
    # a pure function of its arguments, asked once for each
    return load().qs_distill_loss_workspace_bytes(B, V, code)


def distill_loss_workspace_for(logits):
    """A workspace tensor for distill_loss on these logits, or None when the call
    needs none. Reuse it across calls on one stream, for batches of as many rows or
    fewer."""
    n = _workspace_bytes(int(logits.shape[0]), int(logits.shape[1]), _code(logits, "logits"))
    return torch.empty(n, dtype=torch.uint8, device=logits.device) if n else None


def distill_loss(logits, teacher_ids, teacher_values, *, temperature=None, bitmask=None,
                 rest=False, workspace=None):
    """Divergence of each row's tempered, masked softmax from a teacher that is known
    at its top tokens.

    logits [B, V] float32 / bfloat16 (CUDA); teacher_ids int32 [B, K], each token at
    most once, -1 an empty slot; teacher_values float32 [B, K]; temperature float32
    [B] (> 0) or None (1); bitmask int32 [B, >= ceil(V/32)] holding uint32 words, or
    None (slots of illegal tokens count as empty). rest=False: the values are the
    teacher's logits, tempered like the student's and normalised over the listed
    tokens. rest=True: they are its log-probabilities (token_logprobs' top_ids and
    top_logprobs are such lists), and the probability that they leave is compared
    with what the student gives all other tokens. Returns a dict of device tensors:
    loss [B] (NaN on rows whose status is not ROW_OK: leave them out of a sum),
    status [B] and state [B, 8] (for distill_loss_backward). Enqueued on the current
    stream.

    If logits require a gradient, loss carries it (to the logits only; a second
    derivative and forward mode are not available). To capture a training step in a
    graph, drop every eager autograd graph of the same leaves first, as torch asks
    for all backward passes, or capture distill_loss_backward itself.
    """
    shape = _check_inputs(logits, teacher_ids, teacher_values, temperature, bitmask)
    if workspace is not None and (workspace.get_device() != shape[3]
                                  or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{shape[3]}")
    _refuse_tangents(logits, temperature, teacher_values)
    if logits.requires_grad and torch.is_grad_enabled():
        loss, state, status = _DistillLoss.apply(logits, teacher_ids, teacher_values, temperature,
                                                 bitmask, shape, rest, workspace)
    else:
        loss, state, status = _forward(logits, teacher_ids, teacher_values, temperature, bitmask,
                                       shape, rest, workspace)
    return {"loss": loss, "state": state, "status": status}


def _forward(logits, ids, values, temperature, bitmask, shape, rest, workspace):
    lib = load()
    B, V, K, index = shape
    code = _code(logits, "logits")
    # allocations of their own: a loss changed in place (a masked or weighted sum does
    # so) is no change of what the gradient reads. From the teacher's tensors, whose types
    # they have: new_empty with plain sizes takes 1.2 us, empty with a type, a device and a
    # tuple up to 1.7, and short rows are bound by such times
    loss = values.new_empty(B)
    state = values.new_empty(B, STATE)
    status = ids.new_empty(B)
    if workspace is None:
        n = _workspace_bytes(B, V, code)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=logits.device)
    rc = _enqueue(
        lib.qs_distill_loss, index,
        logits.data_ptr(), code, B, V, logits.stride(0), _addr(temperature), _addr(bitmask),
        0 if bitmask is None else bitmask.stride(0), ids.data_ptr(), values.data_ptr(), K,
        1 if rest else 0, loss.data_ptr(), state.data_ptr(), status.data_ptr(), _addr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size())
    if rc:
        _status(rc, "qs_distill_loss")
    return loss, state, status


def distill_loss_backward(logits, teacher_ids, teacher_values, state, status, grad_loss, *,
                          temperature=None, bitmask=None, rest=False, out=None):
    """Gradient of distill_loss with respect to the logits.

    logits, teacher_ids, teacher_values, temperature, bitmask, rest: the forward call's
    inputs; state, status: its outputs; grad_loss float32 [B]. Returns grad_logits
    [B, V] in the logits' dtype (0 on rows whose status is not ROW_OK); out: where to
    write it (it may be logits itself; counted as a change in place, so it must not
    require a gradient).
    """
    B, V, K, index = _check_inputs(logits, teacher_ids, teacher_values, temperature, bitmask)
    _check_vec(status, B, torch.int32, index, "status")
    _check_vec(grad_loss, B, torch.float32, index, "grad_loss")
    if state.dtype is not torch.float32 or state.shape != (B, STATE) \
            or state.get_device() != index or not state.is_contiguous():
        raise ValueError(f"state must be a contiguous float32 tensor [{B}, {STATE}] on "
                         f"cuda:{index}")
    given = out is not None
    if not given:
        out = _padded_rows(B, V, logits.dtype, logits.device)
    elif out.shape != logits.shape or out.dtype is not logits.dtype \
            or out.get_device() != index or out.stride(1) != 1:
        raise ValueError("out must have the logits' shape, dtype and device "
                         "and unit column stride")
    if given:
        _check_out(out)
    _refuse_tangents(logits, temperature, teacher_values, state, grad_loss, out)
    rc = _enqueue(
        load().qs_distill_loss_backward, index,
        logits.data_ptr(), _code(logits, "logits"), B, V, logits.stride(0), _addr(temperature),
        _addr(bitmask), 0 if bitmask is None else bitmask.stride(0), teacher_ids.data_ptr(),
        teacher_values.data_ptr(), K, 1 if rest else 0, state.data_ptr(), status.data_ptr(),
        grad_loss.data_ptr(), out.data_ptr(), out.stride(0))
    if rc:
        _status(rc, "qs_distill_loss_backward")
    if given:
        _wrote(out)
    return out


class _DistillLoss(torch.autograd.Function):
    """distill_loss as a node of torch's graph: loss carries a gradient to the logits."""

    @staticmethod
    def forward(ctx, logits, ids, values, temperature, bitmask, shape, rest, workspace):
        loss, state, status = _forward(logits, ids, values, temperature, bitmask, shape, rest,
                                       workspace)
        ctx.rest = rest
        ctx.save_for_backward(logits, ids, values, temperature, bitmask, state, status)
        ctx.mark_non_differentiable(state, status)
        ctx.set_materialize_grads(False)
        return loss, state, status

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_loss, _state, _status_):
        if g_loss is None:
            return (None,) * 8
        logits, ids, values, temperature, bitmask, state, status = ctx.saved_tensors
        grad = distill_loss_backward(logits, ids, values, state, status, g_loss.contiguous(),
                                     temperature=temperature, bitmask=bitmask, rest=ctx.rest)
        return (grad,) + (None,) * 7
