"""Measured cases of the scoring operators and of the 4-bit output head.

Three operators around the token selection, each with its inputs (`prepare`),
one pass through it (`run`: elementary torch operations where `own` is false,
the framework's entry points where it is true), its least work (`work`) and
its definition in 64 bits (`exact`):

- score: log-probabilities of given tokens under the tempered, masked softmax of
  a row of logits, with the row's entropy and its most probable tokens;
- grad: the gradient of those log-probabilities and of the entropy with respect
  to the logits;
- head: logits of hidden states under an output projection held in 4 bits with
  group scales.
"""

import math

import torch

own = False

ROW_OK, ROW_EMPTY, ROW_ALL_NEG_INF, ROW_NONFINITE = 0, 1, 2, 3

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _score(name, B, V, dtype, G=1, top_n=0, mask=False, temp=False, pad=False):
    return {"name": name, "op": "score", "B": B, "V": V, "dtype": dtype, "G": G, "top_n": top_n,
            "mask": mask, "temp": temp, "pad": pad}


def _grad(name, B, V, dtype, G=1, entropy=False, mask=False, temp=False, pad=False):
    return {"name": name, "op": "grad", "B": B, "V": V, "dtype": dtype, "G": G,
            "entropy": entropy, "mask": mask, "temp": temp, "pad": pad}


def _head(name, B, V, K, group, zeros=False, scale="bf16", out="bf16"):
    return {"name": name, "op": "head", "B": B, "V": V, "K": K, "group": group, "zeros": zeros,
            "scale": scale, "out": out}


def listed():
    return [
        # one row: the log-probability of a single stream's token, a call
        # whose time is its launches
        _score("score row", 1, 32000, "f32"),
        # a serving batch that answers log-probability requests: one token per
        # row under a grammar's legal set, 20 alternatives
        _score("score decode", 256, 151936, "bf16", top_n=20, mask=True),
        # draft tokens scored together: 4 tokens per row, a temperature each
        _score("score draft", 64, 128256, "f32", G=4, top_n=5, temp=True),
        # an odd vocabulary, rows without a legal token, empty slots, the
        # longest list of alternatives
        _score("score ragged", 37, 32003, "bf16", G=3, top_n=64, mask=True, temp=True, pad=True),
        # a long prompt or a rollout's tokens, scored in one call
        _score("score rollout", 2048, 151936, "bf16"),
        # a small training batch
        _grad("grad small", 8, 32000, "f32", entropy=True),
        # masked policy with several tokens per row and padded rows
        _grad("grad ragged", 333, 128259, "bf16", G=4, mask=True, temp=True, pad=True),
        # a policy-gradient step with an entropy bonus
        _grad("grad rollout", 2048, 151936, "bf16", entropy=True),
        # a draft model's head for one stream
        _head("head draft", 1, 32000, 2048, 128),
        # the head of one stream's decode step
        _head("head stream", 1, 151936, 4096, 128),
        # a decode batch, zero points, finer groups, logits kept in 32 bits
        _head("head batch", 16, 128256, 4096, 64, zeros=True, out="f32"),
        # the largest decode batch, a wide model, the finest groups
        _head("head wide", 64, 151936, 8192, 32, scale="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("score", "grad", "head"))
    if op == "head":
        group = rng.choice((32, 64, 128))
        K = group * _log_int(rng, max(1, 256 // group), 8192 // group)
        c = _head("", _log_int(rng, 1, 64), _log_int(rng, 1000, 151936), K, group,
                  zeros=rng.random() < 0.5, scale=rng.choice(("bf16", "f32")),
                  out=rng.choice(("bf16", "f32")))
    else:
        dtype = rng.choice(("bf16", "f32"))
        V = _log_int(rng, 1000, 262144)
        most = (2048 * 151936 * 2) // (V * (2 if dtype == "bf16" else 4))
        B = _log_int(rng, 1, min(2048, most))
        kw = {"G": rng.choice((1, 1, 2, 5)), "mask": rng.random() < 0.4,
              "temp": rng.random() < 0.5, "pad": rng.random() < 0.3}
        if op == "score":
            # alternatives come with batches of a serving step's size
            top_n = rng.choice((0, 1, 7, 20, 64)) if B * V <= 256 * 151936 else 0
            c = _score("", B, V, dtype, top_n=top_n, **kw)
        else:
            c = _grad("", B, V, dtype, entropy=rng.random() < 0.5, **kw)
    del c["name"]
    return c


# --------------------------------------------------------------------------
# Inputs

def _padded(B, V, dtype):
    """[B, V] whose rows start 16-byte aligned, as the selection takes them."""
    step = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.empty((B, -(-V // step) * step), dtype=dtype, device="cuda")[:, :V]


def _words(legal):
    """Packed legal-token words (token i: bit i & 31 of word i >> 5)."""
    B, V = legal.shape
    W = -(-V // 32)
    bits = torch.zeros((B, W * 32), dtype=torch.int64, device=legal.device)
    bits[:, :V] = legal
    words = (bits.view(B, W, 32) << torch.arange(32, device=legal.device)).sum(2)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    B, V = case["B"], case["V"]
    s = {"op": case["op"]}
    if case["op"] == "head":
        K, group = case["K"], case["group"]
        # codes as a checkpoint holds them: two per byte, the earlier column in
        # the low half; weights of about 1/sqrt(K), so logits of a few units
        s["codes"] = torch.randint(0, 256, (V, K // 2), generator=g, device="cuda",
                                   dtype=torch.uint8)
        s["scales"] = ((0.5 + rand(V, K // group)) * (0.6 / math.sqrt(K))).to(
            _DTYPES[case["scale"]])
        s["zeros"] = torch.randint(5, 11, (V, K // group), generator=g, device="cuda",
                                   dtype=torch.uint8) if case["zeros"] else None
        s["hidden"] = randn(B, K).to(torch.bfloat16)
        s["dtype"] = _DTYPES[case["out"]]
        return s
    G = case["G"]
    z = randn(B, V).mul_(3.0)
    logits = _padded(B, V, _DTYPES[case["dtype"]])
    logits.copy_(z)
    s["logits"] = logits
    s["temperature"] = 0.5 + rand(B) if case["temp"] else None
    legal = None
    s["bitmask"] = None
    if case["mask"]:
        legal = rand(B, V) < 0.3
        # some rows' grammar leaves no token at all
        legal[rand(B) < 0.05] = False
        s["bitmask"] = _words(legal)
    # the tokens that were drawn from the same rows, as a rollout holds them
    tokens = torch.empty((B, G), dtype=torch.int32, device="cuda")
    for j in range(G):
        y = z if s["temperature"] is None else z / s["temperature"][:, None]
        y = y - torch.log(-torch.log(rand(B, V).clamp_(1e-30, 1.0 - 2.0 ** -24)))
        if legal is not None:
            y = y.masked_fill_(~legal, -3.0e38)
        tokens[:, j] = y.argmax(1)
    if case["pad"]:
        tokens[rand(B, G) < 0.1] = -1
    s["tokens"] = tokens
    if case["op"] == "score":
        s["top_n"] = case["top_n"]
        return s
    # what the forward pass left: each row's largest legal logit, the log of the
    # sum below it, the entropy and the row status
    x = logits.double()
    T = torch.ones(B, device="cuda") if s["temperature"] is None else s["temperature"]
    if legal is not None:
        x.masked_fill_(~legal, -math.inf)
    s["row_max"] = x.amax(1).float()
    x.sub_(s["row_max"].double()[:, None]).div_(T.double()[:, None])
    e = x.exp()
    S = e.sum(1)
    s["log_sum"] = S.log().float()
    s["status"] = (~torch.isfinite(s["row_max"])).to(torch.int32) * ROW_EMPTY
    # advantages and an entropy bonus, averaged over the batch
    s["grad_logprobs"] = randn(B, G) / B
    s["entropy"] = s["grad_entropy"] = None
    if case["entropy"]:
        x.masked_fill_(e == 0.0, 0.0)
        s["entropy"] = (S.log() - (e.mul_(x)).sum(1) / S).float()
        s["grad_entropy"] = (0.01 + 0.001 * randn(B)) / B
    return s


# --------------------------------------------------------------------------
# One pass

def run(s):
    if own:
        return _run_own(s)
    return {"score": _plain_score, "grad": _plain_grad, "head": _plain_head}[s["op"]](s)


def _run_own(s):
    import top_sampling_vocabs_amd as qs
    if s["op"] == "head":
        return {"logits": qs.head_logits(s["hidden"], s["codes"], s["scales"], s["zeros"],
                                         dtype=s["dtype"])}
    if s["op"] == "grad":
        return {"grad_logits": qs.token_logprobs_backward(
            s["logits"], s["tokens"], s["row_max"], s["log_sum"], s["status"],
            s["grad_logprobs"], temperature=s["temperature"], bitmask=s["bitmask"],
            entropy=s["entropy"], grad_entropy=s["grad_entropy"])}
    return qs.token_logprobs(s["logits"], s["tokens"], temperature=s["temperature"],
                             bitmask=s["bitmask"], entropy=True, top_n=s["top_n"])


def _legal(s):
    B, V = s["logits"].shape
    if s["bitmask"] is None:
        return torch.ones((B, V), dtype=torch.bool, device=s["logits"].device)
    i = torch.arange(V, device=s["logits"].device)
    return (s["bitmask"][:, i >> 5] >> (i & 31)) & 1 == 1


def _plain_score(s):
    legal = _legal(s)
    z = s["logits"].float()
    bad = (legal & ((z != z) | (z == math.inf))).any(1)
    z = torch.where(legal, z, -math.inf)
    top = z.amax(1)
    status = torch.where(top == -math.inf, ROW_ALL_NEG_INF, ROW_OK)
    status = torch.where(bad, ROW_NONFINITE, status)
    status = torch.where(legal.any(1), status, ROW_EMPTY).to(torch.int32)
    ok = status == ROW_OK
    d = z - top[:, None]
    if s["temperature"] is not None:
        d = d / s["temperature"][:, None]
    e = d.exp()
    S = e.sum(1)
    log_sum = S.log()
    entropy = log_sum - (e * torch.where(e > 0, d, 0.0)).sum(1) / S
    tokens = s["tokens"].long()
    lp = d.gather(1, tokens.clamp(min=0)) - log_sum[:, None]
    lp = torch.where(ok[:, None], lp, math.nan)
    out = {"logprobs": torch.where(tokens < 0, 0.0, lp),
           "row_max": torch.where(ok, top, math.nan),
           "log_sum": torch.where(ok, log_sum, math.nan),
           "entropy": torch.where(ok, entropy, math.nan), "status": status}
    n = s["top_n"]
    if n:
        # one ordered whole number per token: larger logit first, then lower id
        V = z.shape[1]
        b = (z + 0.0).view(torch.int32).long()
        key = torch.where(b >= 0, b, -(b & 0x7FFFFFFF))
        key = (key << 32) + (V - 1 - torch.arange(V, device=z.device))
        m = min(n, V)
        ids = V - 1 - (key.topk(m, 1).values & 0xFFFFFFFF)
        best = d.gather(1, ids)
        live = (best > -math.inf) & ok[:, None]
        out["top_ids"] = torch.where(live, ids, -1).to(torch.int32)
        out["top_logprobs"] = torch.where(live, best - log_sum[:, None], -math.inf)
    return out


def _plain_grad(s):
    legal = _legal(s) & (s["status"] == ROW_OK)[:, None]
    d = s["logits"].float() - s["row_max"][:, None]
    if s["temperature"] is not None:
        d = d / s["temperature"][:, None]
    lp = d - s["log_sum"][:, None]
    p = lp.exp()
    tokens = s["tokens"].long()
    g = torch.where(tokens < 0, 0.0, s["grad_logprobs"])
    grad = -p * g.sum(1)[:, None]
    if s["grad_entropy"] is not None:
        grad -= s["grad_entropy"][:, None] * torch.where(p > 0, p * (lp + s["entropy"][:, None]),
                                                         0.0)
    grad.scatter_add_(1, tokens.clamp(min=0), g)
    if s["temperature"] is not None:
        grad = grad / s["temperature"][:, None]
    return {"grad_logits": torch.where(legal, grad, 0.0).to(s["logits"].dtype)}


def _plain_head(s):
    V, half = s["codes"].shape
    groups = s["scales"].shape[1]
    q = torch.stack((s["codes"] & 15, s["codes"] >> 4), 2).view(V, groups, -1).float()
    zero = 8.0 if s["zeros"] is None else s["zeros"].float()[:, :, None]
    w = (q - zero) * s["scales"].float()[:, :, None]
    return {"logits": (s["hidden"].float() @ w.view(V, 2 * half).t()).to(s["dtype"])}


# --------------------------------------------------------------------------
# Least work of a pass

def work(case):
    B, V = case["B"], case["V"]
    if case["op"] == "head":
        K, groups = case["K"], case["K"] // case["group"]
        size = {"bf16": 2, "f32": 4}
        weights = V * (K // 2 + groups * (size[case["scale"]] + int(case["zeros"])))
        return {"bytes": weights + 2 * B * K + size[case["out"]] * B * V, "flops": 2 * B * V * K}
    logits = B * V * (2 if case["dtype"] == "bf16" else 4)
    mask = 4 * B * -(-V // 32) if case["mask"] else 0
    if case["op"] == "score":
        # per token: difference, product, exponential, two sums, one product
        return {"bytes": logits + mask + B * (8 * case["G"] + 8 * case["top_n"] + 20),
                "flops": 6 * B * V}
    # per token: difference, product, exponential, sum, two products
    return {"bytes": 2 * logits + mask + B * (8 * case["G"] + 24), "flops": 6 * B * V}


# --------------------------------------------------------------------------
# The definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    B = case["B"]
    if case["op"] == "head":
        return {"logits": _exact_head(s, case["group"])}
    parts = [(_exact_score if case["op"] == "score" else _exact_grad)(s, slice(a, a + 128))
             for a in range(0, B, 128)]
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_rows(s, rows):
    """Rows' z / T in 64 bits, -inf at illegal tokens, and the temperatures."""
    z = s["logits"][rows].double()
    V = z.shape[1]
    if s["bitmask"] is not None:
        w = s["bitmask"][rows].long().unsqueeze(2) >> torch.arange(32, device=z.device)
        z[(w & 1).flatten(1)[:, :V] == 0] = -math.inf
    T = torch.ones(z.shape[0], dtype=torch.float64, device=z.device) \
        if s["temperature"] is None else s["temperature"][rows].double()
    return z, T


def _exact_score(s, rows):
    z, T = _exact_rows(s, rows)
    dead = (z == -math.inf).all(1)
    nan = torch.full_like(T, math.nan)
    logp = torch.log_softmax(torch.where(dead[:, None], 0.0, z / T[:, None]), 1)
    p = logp.exp()
    top = z.max(1).values
    tokens = s["tokens"][rows].long()
    at = torch.take_along_dim(logp, tokens.clamp(min=0), 1)
    at[dead] = math.nan
    at[tokens < 0] = 0.0
    out = {"logprobs": at, "row_max": torch.where(dead, nan, top),
           "log_sum": torch.where(dead, nan, torch.logsumexp(z / T[:, None], 1) - top / T),
           "entropy": torch.where(dead, nan, -torch.special.xlogy(p, p).sum(1)),
           "status": dead.to(torch.int32)}
    n = s["top_n"]
    if n:
        order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :n]
        lp = torch.take_along_dim(logp, order, 1)
        gone = torch.isinf(torch.take_along_dim(z, order, 1)) | dead[:, None]
        out["top_ids"] = order.masked_fill(gone, -1).to(torch.int32)
        out["top_logprobs"] = lp.masked_fill(gone, -math.inf)
    return out


def _exact_grad(s, rows):
    z, T = _exact_rows(s, rows)
    live = s["status"][rows] == 0
    lp = z / T[:, None] - (s["row_max"][rows].double() / T + s["log_sum"][rows].double())[:, None]
    lp[~live] = -math.inf
    p = lp.exp()
    tokens, g = s["tokens"][rows].long(), s["grad_logprobs"][rows].double()
    g = g * (tokens >= 0)
    out = -p * g.sum(1, keepdim=True)
    if s["grad_entropy"] is not None:
        H, gH = s["entropy"][rows].double(), s["grad_entropy"][rows].double()
        out -= gH[:, None] * (torch.special.xlogy(p, p) + p * torch.where(live, H, 0.0)[:, None])
    r = torch.arange(z.shape[0], device=z.device)[:, None].expand_as(tokens)
    out.index_put_((r, tokens.clamp(min=0)), g, accumulate=True)
    out /= T[:, None]
    out[z == -math.inf] = 0.0
    out[~live] = 0.0
    return {"grad_logits": out}


def _exact_head(s, group):
    codes = s["codes"].to(torch.int16)
    V, K = codes.shape[0], 2 * codes.shape[1]
    h = s["hidden"].double()
    out = torch.empty((h.shape[0], V), dtype=torch.float64, device=h.device)
    for a in range(0, V, 8192):
        c = codes[a:a + 8192]
        w = torch.empty((c.shape[0], K), dtype=torch.float64, device=h.device)
        w[:, 0::2] = (c % 16).double()
        w[:, 1::2] = (c // 16).double()
        if s["zeros"] is None:
            w -= 8.0
        else:
            w -= s["zeros"][a:a + 8192].double().repeat_interleave(group, 1)
        w *= s["scales"][a:a + 8192].double().repeat_interleave(group, 1)
        out[:, a:a + 8192] = h @ w.t()
    return out
