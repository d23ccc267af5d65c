"""Scores of given tokens, their gradient, and the 4-bit output head.

The binding of qs_token_logprobs, qs_token_logprobs_backward and
qs_head_logits. Like the rest of the binding it only marshals arguments; it is
loaded on first use, because it needs torch at import.
"""

import contextlib

import torch

from ._lib import QS_BF16, QS_F32, _check_logits, _check_rowvec, _status, load, sample

_CODES = {torch.float32: QS_F32, torch.bfloat16: QS_BF16}
_SAME_DEVICE = contextlib.nullcontext()


def _code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


def _addr(t):
    """A tensor's address as a C argument (an int; None is NULL)."""
    return None if t is None else t.data_ptr()


def _on(device):
    """Context in which `device` is the current one (kernels launch there)."""
    return _SAME_DEVICE if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)


def _stream(device):
    """The handle of the device's current torch stream (no Stream object made)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _check_device(t, device, name):
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _check_row_inputs(logits, tokens, temperature, bitmask):
    """The forward and the backward call's common inputs: (B, V, G)."""
    B, V = _check_logits(logits, bitmask)
    dev = logits.device
    if bitmask is not None:
        _check_device(bitmask, dev, "bitmask")
    if temperature is not None:
        _check_rowvec(temperature, B, torch.float32, "temperature")
        _check_device(temperature, dev, "temperature")
    if tokens.dtype != torch.int32 or tokens.dim() not in (1, 2) or tokens.shape[0] != B \
            or tokens.device != dev or not tokens.is_contiguous():
        raise ValueError(f"tokens must be a contiguous int32 tensor [B] or [B, G] on {dev}")
    return B, V, tokens.shape[1] if tokens.dim() == 2 else 1


def _padded_rows(B, V, dtype, device):
    """[B, V] uninitialised, rows starting 16 bytes aligned."""
    over = -V % (4 if dtype == torch.float32 else 8)
    t = torch.empty((B, V + over), dtype=dtype, device=device)
    return t[:, :V] if over else t


def token_logprobs_workspace_for(logits, top_n=0):
    """A workspace tensor for token_logprobs on these logits, or None when the
    call needs none. Reuse it across calls on one stream."""
    n = load().qs_token_logprobs_workspace_bytes(int(logits.shape[0]), int(logits.shape[1]),
                                                 _code(logits, "logits"), int(top_n))
    return torch.empty(n, dtype=torch.uint8, device=logits.device) if n else None


def token_logprobs(logits, tokens, *, temperature=None, bitmask=None, entropy=False, top_n=0,
                   workspace=None):
    """Log-probabilities of given tokens under the full tempered, masked softmax.

    logits [B, V] float32 / bfloat16 (CUDA); tokens int32 [B] or [B, G], -1 an
    empty slot (log-probability 0); temperature float32 [B] (> 0) or None (1);
    bitmask int32 [B, >= ceil(V/32)] holding uint32 words, or None. Returns a
    dict of device tensors: logprobs (the shape of tokens), row_max [B],
    log_sum [B], status [B], and if requested entropy [B] (nats), top_ids and
    top_logprobs [B, top_n] (top_n <= 64). Enqueued on the current stream.

    If logits require a gradient, logprobs and entropy carry it (to the logits
    only; a second derivative is not available). To capture a training step in a
    graph, drop every eager autograd graph of the same leaves first, as torch
    asks for all backward passes, or capture token_logprobs_backward itself.
    """
    B, V, G = _check_row_inputs(logits, tokens, temperature, bitmask)
    if workspace is not None:
        _check_device(workspace, logits.device, "workspace")
    if logits.requires_grad and torch.is_grad_enabled():
        keys, *out = _TokenLogprobs.apply(logits, tokens, temperature, bitmask, B, V, G, entropy,
                                          int(top_n), workspace)
        return dict(zip(keys, out))
    return _forward(logits, tokens, temperature, bitmask, B, V, G, entropy, top_n, workspace)


def _forward(logits, tokens, temperature, bitmask, B, V, G, entropy, top_n, workspace):
    lib = load()
    dev = logits.device
    code = _code(logits, "logits")
    lps = torch.empty(tokens.shape, dtype=torch.float32, device=dev)
    # the values per row in one allocation
    row_max, log_sum, status, *ent = torch.empty((4 if entropy else 3, B), dtype=torch.float32,
                                                 device=dev).unbind(0)
    status = status.view(torch.int32)
    out = {"logprobs": lps, "row_max": row_max, "log_sum": log_sum, "status": status}
    if entropy:
        out["entropy"] = ent[0]
    ids = tops = None
    if top_n:
        out["top_ids"] = ids = torch.empty((B, top_n), dtype=torch.int32, device=dev)
        out["top_logprobs"] = tops = torch.empty((B, top_n), dtype=torch.float32, device=dev)
    if workspace is None:
        n = lib.qs_token_logprobs_workspace_bytes(B, V, code, top_n)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    with _on(dev):
        rc = lib.qs_token_logprobs(
            logits.data_ptr(), code, B, V, logits.stride(0), _addr(temperature), _addr(bitmask),
            0 if bitmask is None else bitmask.stride(0), tokens.data_ptr(), G, lps.data_ptr(),
            row_max.data_ptr(), log_sum.data_ptr(), ent[0].data_ptr() if entropy else None,
            top_n, _addr(ids), _addr(tops), status.data_ptr(), _addr(workspace),
            0 if workspace is None else workspace.numel() * workspace.element_size(),
            _stream(dev))
    if rc:
        _status(rc, "qs_token_logprobs")
    return out


def token_logprobs_backward(logits, tokens, row_max, log_sum, status, grad_logprobs, *,
                            temperature=None, bitmask=None, entropy=None, grad_entropy=None,
                            out=None):
    """Gradient of token_logprobs with respect to the logits.

    logits, tokens, temperature, bitmask: the forward call's inputs; row_max,
    log_sum, status (and entropy): its outputs; grad_logprobs float32 in the
    shape of tokens; grad_entropy float32 [B], together with entropy, or None.
    Returns grad_logits [B, V] in the logits' dtype (0 on rows whose status is
    not ROW_OK); out: where to write it (it may be logits itself).
    """
    B, V, G = _check_row_inputs(logits, tokens, temperature, bitmask)
    dev = logits.device
    if (entropy is None) != (grad_entropy is None):
        raise ValueError("entropy and grad_entropy go together")
    for t, dtype, name in ((row_max, torch.float32, "row_max"), (log_sum, torch.float32, "log_sum"),
                           (status, torch.int32, "status"), (entropy, torch.float32, "entropy"),
                           (grad_entropy, torch.float32, "grad_entropy")):
        if t is not None or name not in ("entropy", "grad_entropy"):
            _check_rowvec(t, B, dtype, name)
            _check_device(t, dev, name)
    if grad_logprobs.shape != tokens.shape or grad_logprobs.dtype != torch.float32 \
            or grad_logprobs.device != dev or not grad_logprobs.is_contiguous():
        raise ValueError("grad_logprobs must be a contiguous float32 tensor in the shape of "
                         f"tokens on {dev}")
    if out is None:
        out = _padded_rows(B, V, logits.dtype, dev)
    elif out.shape != logits.shape or out.dtype != logits.dtype or out.device != dev \
            or out.stride(1) != 1:
        raise ValueError("out must have the logits' shape, dtype and device "
                         "and unit column stride")
    with _on(dev):
        rc = load().qs_token_logprobs_backward(
            logits.data_ptr(), _code(logits, "logits"), B, V, logits.stride(0), _addr(temperature),
            _addr(bitmask), 0 if bitmask is None else bitmask.stride(0), tokens.data_ptr(), G,
            row_max.data_ptr(), log_sum.data_ptr(), status.data_ptr(), grad_logprobs.data_ptr(),
            _addr(entropy), _addr(grad_entropy), out.data_ptr(), out.stride(0), _stream(dev))
    if rc:
        _status(rc, "qs_token_logprobs_backward")
    return out


class _TokenLogprobs(torch.autograd.Function):
    """token_logprobs as a node of torch's graph: logprobs and entropy carry a
    gradient to the logits."""

    @staticmethod
    def forward(ctx, logits, tokens, temperature, bitmask, B, V, G, entropy, top_n, workspace):
        out = _forward(logits, tokens, temperature, bitmask, B, V, G, entropy, top_n, workspace)
        ctx.keys = tuple(out)
        ctx.save_for_backward(logits, tokens, temperature, bitmask, out["row_max"],
                              out["log_sum"], out["status"], out.get("entropy"))
        ctx.mark_non_differentiable(*(v for k, v in out.items()
                                      if k not in ("logprobs", "entropy")))
        ctx.set_materialize_grads(False)
        return (ctx.keys, *out.values())

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _keys, *grads):
        logits, tokens, temperature, bitmask, row_max, log_sum, status, ent = ctx.saved_tensors
        g = dict(zip(ctx.keys, grads))
        g_lp, g_ent = g["logprobs"], g.get("entropy")
        if g_lp is None and g_ent is None:
            return (None,) * 10
        if g_lp is None:
            g_lp = torch.zeros(tokens.shape, dtype=torch.float32, device=tokens.device)
        grad = token_logprobs_backward(
            logits, tokens, row_max, log_sum, status, g_lp.contiguous(),
            temperature=temperature, bitmask=bitmask,
            entropy=None if g_ent is None else ent,
            grad_entropy=None if g_ent is None else g_ent.contiguous())
        return (grad,) + (None,) * 9


def head_logits(hidden, codes, scales, zeros=None, *, dtype=None, out=None):
    """Logits of hidden states under an output projection held in 4 bits.

    hidden bfloat16 [B, K]; codes uint8 [V, K/2], two codes a byte, the even
    column in the low half; scales float32 / bfloat16 [V, K/group], group 32, 64
    or 128; zeros uint8 [V, K/group] or None (8). Weight [v, k] is
    (code - zero) * scale. Returns logits [B, V] in `dtype` (bfloat16 unless
    given) with rows laid out as the selection reads them; out: where to write
    them. Enqueued on the current stream. Inference only: tensors that require
    a gradient are refused.
    """
    if hidden.dim() != 2 or not hidden.is_cuda or hidden.dtype != torch.bfloat16 \
            or hidden.stride(1) != 1:
        raise ValueError("hidden must be a bfloat16 CUDA tensor [B, K] with unit column stride")
    dev = hidden.device
    B, K = hidden.shape
    if codes.dim() != 2 or codes.dtype != torch.uint8 or codes.shape[1] * 2 != K \
            or codes.stride(1) != 1 or codes.device != dev:
        raise ValueError(f"codes must be a uint8 tensor [V, K/2] with unit column stride on {dev}")
    V = codes.shape[0]
    groups = scales.shape[1] if scales.dim() == 2 else 0
    if groups < 1 or scales.shape[0] != V or K % groups or K // groups not in (32, 64, 128) \
            or scales.stride(1) != 1 or scales.device != dev:
        raise ValueError("scales must be [V, K/group] with group 32, 64 or 128 "
                         f"and unit column stride on {dev}")
    if zeros is not None and (zeros.shape != scales.shape or zeros.dtype != torch.uint8
                              or zeros.stride(1) != 1 or zeros.device != dev):
        raise ValueError(f"zeros must be a uint8 tensor in the shape of scales on {dev}")
    if (hidden.requires_grad or scales.requires_grad) and torch.is_grad_enabled():
        raise ValueError("head_logits has no gradient: call it under torch.no_grad() "
                         "or on detached tensors")
    if out is None:
        out = _padded_rows(B, V, dtype or torch.bfloat16, dev)
    elif out.shape != (B, V) or out.stride(1) != 1 or out.device != dev \
            or (dtype is not None and out.dtype != dtype):
        raise ValueError("out must be [B, V] in the asked dtype with unit column stride "
                         f"on {dev}")
    with _on(dev):
        rc = load().qs_head_logits(
            hidden.data_ptr(), B, K, hidden.stride(0) if B > 1 else K, codes.data_ptr(), V, codes.stride(0),
            scales.data_ptr(), _code(scales, "scales"), scales.stride(0), _addr(zeros),
            0 if zeros is None else zeros.stride(0), K // groups, out.data_ptr(),
            _code(out, "out"), out.stride(0), _stream(dev))
    if rc:
        _status(rc, "qs_head_logits")
    return out


def sample_hidden(hidden, codes, scales, zeros, temperature, top_k, top_p, bitmask=None, *,
                  dtype=None, logits=None, **options):
    """sample() from hidden states: head_logits into `logits` (a buffer [B, V];
    made per call when omitted), then the selection, on the current stream.
    options: sample()'s keyword arguments. The result holds the logits too."""
    z = head_logits(hidden, codes, scales, zeros, dtype=dtype, out=logits)
    out = sample(z, temperature, top_k, top_p, bitmask, **options)
    out["logits"] = z
    return out
