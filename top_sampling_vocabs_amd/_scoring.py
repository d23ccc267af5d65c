"""Scores of given tokens, their gradient, and the 4-bit output head.

The binding of qs_token_logprobs, qs_token_logprobs_backward and
qs_head_logits. Like the rest of the binding it only marshals arguments; it is
loaded on first use, because it needs torch at import.
"""

import torch
from torch.autograd import forward_ad

from ._lib import QS_BF16, QS_F32, _check_logits, _status, load, sample

_CODES = {torch.float32: QS_F32, torch.bfloat16: QS_BF16}
# what torch.cuda's own calls are made of, without their checks and without a Stream
# object; those themselves where a torch does not have these
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


def _addr(t):
    """A tensor's address as a C argument (an int; None is NULL)."""
    return None if t is None else t.data_ptr()


def _enqueue(call, index, *args):
    """call(*args, stream) on the current torch stream of device `index`, with that
    device the current one (kernels launch there)."""
    if _current_device() == index:
        return call(*args, _current_stream(index))
    with torch.cuda.device(index):
        return call(*args, _current_stream(index))


def _refuse_tangents(*tensors):
    """Forward-mode tangents would be dropped without a word: refused. (Outside a
    dual level no tensor has one; a torch that does not say is asked for each.)"""
    if getattr(forward_ad, "_current_level", 0) < 0:
        return
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError("tangents of forward-mode differentiation are not carried")


def _check_out(out):
    """An output buffer of the caller's: written without a node of torch's graph, so
    it cannot be one that a gradient flows through."""
    if out.requires_grad and torch.is_grad_enabled():
        raise ValueError("an output buffer must not require a gradient: call under "
                         "torch.no_grad() or with a detached tensor")


def _wrote(out):
    """Counts a launched kernel's writes into the caller's tensor as a change in
    place: a graph that saved the tensor reports it instead of reading it."""
    torch.autograd.graph.increment_version(out)


def _check_vec(t, B, dtype, index, name):
    # one test a property, the cheap ones first: most calls here are small
    if t is None or t.dtype is not dtype or t.dim() != 1 or t.size(0) != B \
            or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape [{B}] and {dtype} on "
                         f"cuda:{index}")


def _check_row_inputs(logits, tokens, temperature, bitmask):
    """The forward and the backward call's common inputs: (B, V, G, device index)."""
    B, V = _check_logits(logits, bitmask)
    index = logits.get_device()
    if bitmask is not None and bitmask.get_device() != index:
        raise ValueError(f"bitmask must be on cuda:{index}, got {bitmask.device}")
    if temperature is not None:
        _check_vec(temperature, B, torch.float32, index, "temperature")
    n = tokens.dim()
    if tokens.dtype is not torch.int32 or n not in (1, 2) or tokens.size(0) != B \
            or tokens.get_device() != index or not tokens.is_contiguous():
        raise ValueError("tokens must be a contiguous int32 tensor [B] or [B, G] on "
                         f"cuda:{index}")
    return B, V, tokens.size(1) if n == 2 else 1, index


def _padded_rows(B, V, dtype, device):
    """[B, V] uninitialised, rows starting 16 bytes aligned."""
    width = V + -V % (4 if dtype is torch.float32 else 8)
    t = torch.empty((B, width), dtype=dtype, device=device)
    return t if width == V else t.as_strided((B, V), (width, 1))


def token_logprobs_workspace_for(logits, top_n=0):
    """A workspace tensor for token_logprobs on these logits, or None when the
    call needs none. Reuse it across calls on one stream, for batches of as many
    rows or fewer."""
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
    only; a second derivative and forward mode are not available). To capture a
    training step in a graph, drop every eager autograd graph of the same leaves
    first, as torch asks for all backward passes, or capture
    token_logprobs_backward itself.
    """
    shape = _check_row_inputs(logits, tokens, temperature, bitmask)
    if workspace is not None and (workspace.get_device() != shape[3]
                                  or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{shape[3]}")
    _refuse_tangents(logits, temperature)
    if logits.requires_grad and torch.is_grad_enabled():
        keys, *out = _TokenLogprobs.apply(logits, tokens, temperature, bitmask, shape, entropy,
                                          int(top_n), workspace)
        return dict(zip(keys, out))
    return _forward(logits, tokens, temperature, bitmask, shape, entropy, top_n, workspace)


def _forward(logits, tokens, temperature, bitmask, shape, entropy, top_n, workspace):
    lib = load()
    dev = logits.device
    B, V, G, index = shape
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
    rc = _enqueue(
        lib.qs_token_logprobs, index,
        logits.data_ptr(), code, B, V, logits.stride(0), _addr(temperature), _addr(bitmask),
        0 if bitmask is None else bitmask.stride(0), tokens.data_ptr(), G, lps.data_ptr(),
        row_max.data_ptr(), log_sum.data_ptr(), ent[0].data_ptr() if entropy else None,
        top_n, _addr(ids), _addr(tops), status.data_ptr(), _addr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size())
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
    not ROW_OK); out: where to write it (it may be logits itself; counted as a
    change in place, so it must not require a gradient).
    """
    B, V, G, index = _check_row_inputs(logits, tokens, temperature, bitmask)
    if (entropy is None) != (grad_entropy is None):
        raise ValueError("entropy and grad_entropy go together")
    _check_vec(row_max, B, torch.float32, index, "row_max")
    _check_vec(log_sum, B, torch.float32, index, "log_sum")
    _check_vec(status, B, torch.int32, index, "status")
    if entropy is not None:
        _check_vec(entropy, B, torch.float32, index, "entropy")
        _check_vec(grad_entropy, B, torch.float32, index, "grad_entropy")
    if grad_logprobs.dtype is not torch.float32 or grad_logprobs.shape != tokens.shape \
            or grad_logprobs.get_device() != index or not grad_logprobs.is_contiguous():
        raise ValueError("grad_logprobs must be a contiguous float32 tensor in the shape of "
                         f"tokens on cuda:{index}")
    given = out is not None
    if not given:
        out = _padded_rows(B, V, logits.dtype, logits.device)
    elif out.shape != logits.shape or out.dtype is not logits.dtype \
            or out.get_device() != index or out.stride(1) != 1:
        raise ValueError("out must have the logits' shape, dtype and device "
                         "and unit column stride")
    if given:
        _check_out(out)
    _refuse_tangents(logits, temperature, row_max, log_sum, grad_logprobs, entropy, grad_entropy,
                     out)
    rc = _enqueue(
        load().qs_token_logprobs_backward, index,
        logits.data_ptr(), _code(logits, "logits"), B, V, logits.stride(0), _addr(temperature),
        _addr(bitmask), 0 if bitmask is None else bitmask.stride(0), tokens.data_ptr(), G,
        row_max.data_ptr(), log_sum.data_ptr(), status.data_ptr(), grad_logprobs.data_ptr(),
        _addr(entropy), _addr(grad_entropy), out.data_ptr(), out.stride(0))
    if rc:
        _status(rc, "qs_token_logprobs_backward")
    if given:
        _wrote(out)
    return out


class _TokenLogprobs(torch.autograd.Function):
    """token_logprobs as a node of torch's graph: logprobs and entropy carry a
    gradient to the logits."""

    @staticmethod
    def forward(ctx, logits, tokens, temperature, bitmask, shape, entropy, top_n, workspace):
        out = _forward(logits, tokens, temperature, bitmask, shape, entropy, top_n, workspace)
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
            return (None,) * 8
        if g_lp is None:
            g_lp = torch.zeros(tokens.shape, dtype=torch.float32, device=tokens.device)
        grad = token_logprobs_backward(
            logits, tokens, row_max, log_sum, status, g_lp.contiguous(),
            temperature=temperature, bitmask=bitmask,
            entropy=None if g_ent is None else ent,
            grad_entropy=None if g_ent is None else g_ent.contiguous())
        return (grad,) + (None,) * 7


def head_logits(hidden, codes, scales, zeros=None, *, dtype=None, out=None):
    """Logits of hidden states under an output projection held in 4 bits.

    hidden bfloat16 [B, K]; codes uint8 [V, K/2], two codes a byte, the even
    column in the low half; scales float32 / bfloat16 [V, K/group], group 32, 64
    or 128; zeros uint8 [V, K/group] or None (8). Weight [v, k] is
    (code - zero) * scale. Returns logits [B, V] in `dtype` (bfloat16 unless
    given) with rows laid out as the selection reads them; out: where to write
    them (counted as a change in place). Enqueued on the current stream. Inference
    only: tensors that require a gradient or carry a tangent are refused.
    """
    if hidden.dtype is not torch.bfloat16 or hidden.dim() != 2 or not hidden.is_cuda \
            or hidden.stride(1) != 1:
        raise ValueError("hidden must be a bfloat16 CUDA tensor [B, K] with unit column stride")
    index = hidden.get_device()
    B, K = hidden.shape
    if codes.dtype is not torch.uint8 or codes.dim() != 2 or codes.size(1) * 2 != K \
            or codes.stride(1) != 1 or codes.get_device() != index:
        raise ValueError("codes must be a uint8 tensor [V, K/2] with unit column stride on "
                         f"cuda:{index}")
    V = codes.size(0)
    groups = scales.size(1) if scales.dim() == 2 else 0
    if groups < 1 or scales.size(0) != V or K % groups or K // groups not in (32, 64, 128) \
            or scales.stride(1) != 1 or scales.get_device() != index:
        raise ValueError("scales must be [V, K/group] with group 32, 64 or 128 "
                         f"and unit column stride on cuda:{index}")
    if zeros is not None and (zeros.dtype is not torch.uint8 or zeros.shape != scales.shape
                              or zeros.stride(1) != 1 or zeros.get_device() != index):
        raise ValueError(f"zeros must be a uint8 tensor in the shape of scales on cuda:{index}")
    if (hidden.requires_grad or scales.requires_grad) and torch.is_grad_enabled():
        raise ValueError("head_logits has no gradient: call it under torch.no_grad() "
                         "or on detached tensors")
    _refuse_tangents(hidden, scales, out)
    given = out is not None
    if not given:
        out = _padded_rows(B, V, dtype or torch.bfloat16, hidden.device)
    elif out.shape != (B, V) or out.stride(1) != 1 or out.get_device() != index \
            or (dtype is not None and out.dtype is not dtype):
        raise ValueError("out must be [B, V] in the asked dtype with unit column stride "
                         f"on cuda:{index}")
    if given:
        _check_out(out)
    rc = _enqueue(
        load().qs_head_logits, index,
        hidden.data_ptr(), B, K, hidden.stride(0) if B > 1 else K, codes.data_ptr(), V,
        codes.stride(0), scales.data_ptr(), _code(scales, "scales"), scales.stride(0),
        _addr(zeros), 0 if zeros is None else zeros.stride(0), K // groups, out.data_ptr(),
        _code(out, "out"), out.stride(0))
    if rc:
        _status(rc, "qs_head_logits")
    if given:
        _wrote(out)
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
