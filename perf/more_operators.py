"""Measured cases of distillation from a teacher's top tokens, of its gradient, and
of low-rank adapters beside the output projection.

Three operators around the token selection, each with its inputs (`prepare`),
one pass through it (`run`: elementary torch operations where `own` is false,
the framework's entry points where it is true), its least work (`work`) and
its definition in 64 bits (`exact`):

- distill: the divergence of a student's tempered, masked softmax from a teacher
  that is known at its top tokens only;
- grad: the gradient of that loss with respect to the student's logits;
- adapters: what low-rank adapters add to the logits of a batch whose rows use
  adapters of their own.
"""

import math

import torch

own = False

ROW_OK, ROW_EMPTY, ROW_ALL_NEG_INF, ROW_NONFINITE, ROW_BAD_PARAM = 0, 1, 2, 3, 4

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _distill(name, B, V, dtype, K, op="distill", rest=False, mask=False, temp=False, pad=False):
    return {"name": name, "op": op, "B": B, "V": V, "dtype": dtype, "K": K, "rest": rest,
            "mask": mask, "temp": temp, "pad": pad}


def _adapters(name, B, V, K, rank, held, used, without=0, dtype="bf16", scale=True):
    """`held` adapters in memory, `used` of them by the batch, `without` rows with none."""
    return {"name": name, "op": "adapters", "B": B, "V": V, "K": K, "rank": rank, "held": held,
            "used": used, "without": without, "dtype": dtype, "scale": scale}


def listed():
    return [
        # one row: a call whose time is its launches
        _distill("distill row", 1, 32000, "f32", 20),
        # a small batch in 32 bits, the rest of the teacher's mass as one more
        # outcome, a temperature each
        _distill("distill batch", 64, 128256, "f32", 50, rest=True, temp=True),
        # an odd vocabulary, a grammar's legal set, short and empty lists
        _distill("distill ragged", 37, 32003, "bf16", 33, rest=True, mask=True, temp=True,
                 pad=True),
        # the tokens of a training step against a teacher's 64 stored tokens
        _distill("distill rollout", 2048, 151936, "bf16", 64, rest=True),
        # a small training batch
        _distill("grad small", 8, 32000, "f32", 20, op="grad"),
        # masked rows of an odd length, long lists, padded positions
        _distill("grad ragged", 333, 128259, "bf16", 256, op="grad", rest=True, mask=True,
                 temp=True, pad=True),
        # the training step's gradient, teacher and student tempered alike
        _distill("grad rollout", 2048, 151936, "bf16", 64, op="grad", temp=True),
        # a draft model's head, two streams with small adapters
        _adapters("adapters draft", 2, 32000, 2048, 8, held=4, used=2),
        # one stream's decode step
        _adapters("adapters stream", 1, 151936, 4096, 16, held=8, used=1),
        # a decode batch, every request with its own adapter, logits in 32 bits
        _adapters("adapters batch", 16, 128256, 4096, 32, held=16, used=16, dtype="f32"),
        # the largest decode batch on three adapters of high rank, some rows
        # without one
        _adapters("adapters shared", 64, 151936, 4096, 64, held=3, used=3, without=10),
        # the largest decode batch of a wide model, every request with its own
        _adapters("adapters wide", 64, 151936, 8192, 32, held=64, used=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("distill", "grad", "adapters"))
    if op == "adapters":
        B, V = _log_int(rng, 1, 64), _log_int(rng, 1000, 151936)
        rank = 8 * _log_int(rng, 1, 16)
        most = (64 * 151936 * 32) // (V * rank)
        without = min(rng.choice((0, 0, 1, B // 4)), B - 1)
        used = min(B - without, _log_int(rng, 1, 64), most)
        held = min(used + rng.choice((1, 2, 5)), most + 1)
        c = _adapters("", B, V, 32 * _log_int(rng, 8, 256), rank, held=held, used=used,
                      without=without, dtype=rng.choice(("bf16", "f32")), scale=rng.random() < 0.7)
    else:
        dtype = rng.choice(("bf16", "f32"))
        V = _log_int(rng, 1000, 262144)
        most = (2048 * 151936 * 2) // (V * (2 if dtype == "bf16" else 4))
        c = _distill("", _log_int(rng, 1, min(2048, most)), V, dtype, _log_int(rng, 1, 512), op=op,
                     rest=rng.random() < 0.5, mask=rng.random() < 0.4, temp=rng.random() < 0.5,
                     pad=rng.random() < 0.3)
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

    B, V, K = case["B"], case["V"], case["K"]
    dtype = _DTYPES[case["dtype"]]
    s = {"op": case["op"]}
    if case["op"] == "adapters":
        held, used, rank = case["held"], case["used"], case["rank"]
        # the shared projection's logits, and where the adapted ones go
        s["logits"] = _padded(B, V, dtype)
        s["logits"].copy_(randn(B, V).mul_(3.0))
        s["out"] = _padded(B, V, dtype)
        s["hidden"] = randn(B, K).to(torch.bfloat16)
        # both factors as training leaves them: adapted logits move by about one unit
        s["down"] = torch.empty((held, rank, K), dtype=torch.bfloat16, device="cuda").normal_(
            0.0, 1.0 / math.sqrt(K), generator=g)
        s["up"] = torch.empty((held, V, rank), dtype=torch.bfloat16, device="cuda").normal_(
            0.0, 1.0 / math.sqrt(rank), generator=g)
        s["scale"] = 0.5 + rand(held) if case["scale"] else None
        # each used adapter once, the other rows any of them, some rows none
        ids = torch.randperm(held, generator=g, device="cuda")[:used]
        index = torch.full((B,), -1, dtype=torch.int64, device="cuda")
        rows = B - case["without"]
        if rows:
            more = torch.randint(0, used, (rows - used,), generator=g, device="cuda")
            index[:rows] = torch.cat((ids, ids[more]))
        s["index"] = index[torch.randperm(B, generator=g, device="cuda")].to(torch.int32)
        return s
    z = randn(B, V).mul_(3.0)
    s["logits"] = _padded(B, V, dtype)
    s["logits"].copy_(z)
    s["temperature"] = 0.5 + 1.5 * rand(B) if case["temp"] else None
    # a teacher that agrees with its student in part
    z.mul_(0.8).add_(randn(B, V).mul_(1.5))
    s["bitmask"] = None
    if case["mask"]:
        legal = rand(B, V) < 0.3
        # some rows' grammar leaves no token at all
        legal[rand(B) < 0.05] = False
        s["bitmask"] = _words(legal)
        z.masked_fill_(~legal, -math.inf)
        del legal
    top = z.topk(min(K, V), 1)
    ids, values = top.indices, top.values
    if case["rest"]:
        # stored log-probabilities of the tempered teacher
        y = z if s["temperature"] is None else z / s["temperature"][:, None]
        values = torch.where(values > -math.inf, y.gather(1, ids) - y.logsumexp(1)[:, None],
                             -math.inf)
        del y
    ids = torch.where(values > -math.inf, ids, -1)
    if case["pad"]:
        # lists shorter than the longest, and positions without any
        n = (rand(B) * 2.0 * K).long()
        n[rand(B) < 0.1] = 0
        gone = torch.arange(ids.shape[1], device="cuda") >= n[:, None]
        ids, values = ids.masked_fill(gone, -1), values.masked_fill(gone, -math.inf)
    s["ids"], s["values"], s["rest"] = ids.to(torch.int32), values.contiguous(), case["rest"]
    if case["op"] == "distill":
        return s
    # what the forward pass left, and the weights of the rows' losses
    s.update(_plain_distill(s))
    del s["loss"]
    s["grad_loss"] = (0.5 + rand(B)) / B
    return s


# --------------------------------------------------------------------------
# One pass

def run(s):
    if own:
        return _run_own(s)
    return {"distill": _plain_distill, "grad": _plain_grad, "adapters": _plain_adapters}[s["op"]](s)


def _run_own(s):
    import top_sampling_vocabs_amd as qs
    if s["op"] == "adapters":
        status = qs.apply_adapters(s["logits"], s["hidden"], s["down"], s["up"], s["index"],
                                   s["scale"], out=s["out"])
        return {"logits": s["out"], "status": status}
    if s["op"] == "grad":
        return {"grad_logits": qs.distill_loss_backward(
            s["logits"], s["ids"], s["values"], s["state"], s["status"], s["grad_loss"],
            temperature=s["temperature"], bitmask=s["bitmask"], rest=s["rest"])}
    return qs.distill_loss(s["logits"], s["ids"], s["values"], temperature=s["temperature"],
                           bitmask=s["bitmask"], rest=s["rest"])


def _legal(s):
    B, V = s["logits"].shape
    if s["bitmask"] is None:
        return torch.ones((B, V), dtype=torch.bool, device=s["logits"].device)
    i = torch.arange(V, device=s["logits"].device)
    return (s["bitmask"][:, i >> 5] >> (i & 31)) & 1 == 1


def _listed(s, legal):
    """The slots whose tokens are legal, their tokens, and every token's place in them."""
    ids = s["ids"].long().clamp(min=0)
    live = (s["ids"] >= 0) & legal.gather(1, ids)
    hit = torch.zeros(legal.shape, dtype=torch.int8, device=legal.device)
    hit.scatter_add_(1, ids, live.to(torch.int8))
    return ids, live, hit > 0


def _temperature(s):
    return torch.ones(len(s["logits"]), device="cuda") if s["temperature"] is None \
        else s["temperature"]


def _plain_distill(s):
    legal, T = _legal(s), _temperature(s)
    z = s["logits"].float()
    bad = (legal & ((z != z) | (z == math.inf))).any(1)
    any_legal = legal.any(1)
    z = torch.where(legal, z, -math.inf)
    ids, live, hit = _listed(s, legal)
    top = z.amax(1)
    status = torch.where(top == -math.inf, ROW_ALL_NEG_INF, ROW_OK)
    status = torch.where(bad, ROW_NONFINITE, status)
    status = torch.where(any_legal, status, ROW_EMPTY).to(torch.int32)
    ok = status == ROW_OK
    mine = z.gather(1, ids)
    # the sums over the whole row in 32 bits, what a row has of them in 64
    log_sum = ((z - top[:, None]) / T[:, None]).exp().sum(1).double().log()
    z = torch.where(hit, -math.inf, z)
    rest_top = z.amax(1)
    there = rest_top > -math.inf
    rest_top = torch.where(there, rest_top, 0.0)
    rest_log = ((z - rest_top[:, None]) / T[:, None]).exp().sum(1).double().log()
    T, top = T.double(), top.double()
    log_p = (mine.double() - top[:, None]) / T[:, None] - log_sum[:, None]
    t = torch.where(live, s["values"], -math.inf).double()
    t_max = torch.zeros_like(T)
    t_log = torch.zeros_like(T)
    if s["rest"]:
        log_q = t
        q_rest = torch.where(there, (1.0 - t.exp().sum(1)).clamp(min=0.0), 0.0)
    else:
        t_max = t.amax(1)
        t_max = torch.where(t_max > -math.inf, t_max, 0.0)
        d = (t - t_max[:, None]) / T[:, None]
        n = d.exp().sum(1)
        t_log = torch.where(n > 0, n.log(), 0.0)
        log_q = d - t_log[:, None]
        q_rest = torch.zeros_like(T)
    q = log_q.exp()
    log_rest = (rest_top.double() - top) / T + rest_log - log_sum
    mass = q.sum(1) + q_rest
    loss = torch.where(q > 0, q * (log_q - log_p), 0.0).sum(1) \
        + torch.where(q_rest > 0, q_rest * (q_rest.log() - log_rest), 0.0)
    rest_grad = torch.where(there, mass * log_rest.exp() - q_rest, 0.0)
    state = torch.stack((top, log_sum, rest_top.double(), torch.where(there, rest_log, 0.0),
                         rest_grad, t_max, t_log, mass - 1.0), 1)
    return {"loss": torch.where(ok, loss, math.nan).float(),
            "state": torch.where(ok[:, None], state, math.nan).float(), "status": status}


def _plain_grad(s):
    T, state = _temperature(s), s["state"]
    legal = _legal(s)
    ok = s["status"] == ROW_OK
    ids, live, hit = _listed(s, legal)
    z = s["logits"].float()
    by = s["grad_loss"].double() / T.double()
    # the listed tokens in 64 bits: what teacher and student agree on cancels
    x = state.double()
    log_p = (z.gather(1, ids).double() - x[:, :1]) / T.double()[:, None] - x[:, 1:2]
    t = torch.where(live, s["values"], -math.inf).double()
    log_q = t if s["rest"] else (t - x[:, 5:6]) / T.double()[:, None] - x[:, 6:7]
    mine = x[:, 7:] + (1.0 + x[:, 7:]) * torch.expm1(log_p) - torch.expm1(log_q)
    mine = torch.where(live, by[:, None] * mine, 0.0)
    w = ((z - state[:, 2:3]) / T[:, None] - state[:, 3:4]).exp()
    grad = torch.where(hit, 0.0, w * (by * x[:, 4]).float()[:, None])
    grad.scatter_add_(1, ids, mine.float())
    return {"grad_logits": torch.where(legal & ok[:, None], grad, 0.0).to(s["logits"].dtype)}


def _plain_adapters(s):
    index = s["index"].long()
    a = index.clamp(min=0)
    u = torch.bmm(s["down"][a].float(), s["hidden"].float()[:, :, None])
    if s["scale"] is not None:
        u = u * s["scale"][a][:, None, None]
    z = s["logits"].float()
    moved = z + torch.bmm(s["up"][a].float(), u)[:, :, 0]
    return {"logits": torch.where((index >= 0)[:, None], moved, z).to(s["logits"].dtype),
            "status": torch.zeros_like(s["index"])}


# --------------------------------------------------------------------------
# Least work of a pass

def work(case):
    B, V, K = case["B"], case["V"], case["K"]
    size = {"bf16": 2, "f32": 4}[case["dtype"]]
    if case["op"] == "adapters":
        rank, rows = case["rank"], B - case["without"]
        return {"bytes": 2 * B * V * size + 2 * B * K + 2 * case["used"] * rank * (K + V) + 12 * B,
                "flops": 2 * rows * rank * (K + V)}
    logits = B * V * size
    mask = 4 * B * -(-V // 32) if case["mask"] else 0
    # per token: difference, product, exponential, sum (the gradient: two products)
    return {"bytes": logits * (1 if case["op"] == "distill" else 2) + mask + B * (8 * K + 44),
            "flops": 4 * B * V}


# --------------------------------------------------------------------------
# The definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    B = case["B"]
    if case["op"] == "adapters":
        return {"logits": torch.stack([_exact_adapted(s, b) for b in range(B)]),
                "status": torch.zeros_like(s["index"])}
    rows = _exact_loss if case["op"] == "distill" else _exact_grad
    parts = [rows(s, slice(a, a + 128)) for a in range(0, B, 128)]
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_rows(s, rows):
    """z / T with -inf at illegal tokens, T, and the teacher's values over the whole
    vocabulary (-inf where none is known), all in 64 bits; which tokens are known."""
    z = s["logits"][rows].double()
    n, V = z.shape
    illegal = torch.zeros((n, V), dtype=torch.bool, device=z.device)
    if s["bitmask"] is not None:
        w = s["bitmask"][rows].long().unsqueeze(2) >> torch.arange(32, device=z.device)
        illegal = (w & 1).flatten(1)[:, :V] == 0
        z[illegal] = -math.inf
    T = torch.ones(n, dtype=torch.float64, device=z.device) if s["temperature"] is None \
        else s["temperature"][rows].double()
    # one place more than the vocabulary takes the empty slots
    to = torch.where(s["ids"][rows] < 0, V, s["ids"][rows]).long()
    teacher = torch.full((n, V + 1), -math.inf, dtype=torch.float64, device=z.device)
    teacher.scatter_(1, to, s["values"][rows].double())
    known = torch.zeros((n, V + 1), dtype=torch.bool, device=z.device)
    known.scatter_(1, to, True)
    teacher, known = teacher[:, :V], known[:, :V] & ~illegal
    return z / T[:, None], z, T, teacher.masked_fill(~known, -math.inf), known


def _exact_loss(s, rows):
    y, z, T, teacher, known = _exact_rows(s, rows)
    dead = (z == -math.inf).all(1)
    total = torch.logsumexp(y, 1)
    others = y.masked_fill(known, -math.inf)
    rest_max = z.masked_fill(known, -math.inf).amax(1)
    there = rest_max > -math.inf
    rest_max = torch.where(there, rest_max, 0.0)
    rest_total = torch.logsumexp(others, 1)
    if s["rest"]:
        q = teacher.exp()
        q_rest = torch.where(there, torch.relu(1.0 - q.sum(1)), 0.0)
        t_max = t_log = torch.zeros_like(T)
    else:
        some = (teacher > -math.inf).any(1)
        t_max = torch.where(some, teacher.amax(1), 0.0)
        t_log = torch.where(some, torch.logsumexp(teacher / T[:, None], 1) - t_max / T, 0.0)
        q = (teacher / T[:, None] - (t_log + t_max / T)[:, None]).exp()
        q_rest = torch.zeros_like(T)
    p_rest = (rest_total - total).exp()
    cross = torch.where(q > 0, q * (total[:, None] - y), 0.0).sum(1)
    loss = torch.special.xlogy(q, q).sum(1) + cross + torch.where(
        q_rest > 0, torch.special.xlogy(q_rest, q_rest) - q_rest * (rest_total - total), 0.0)
    mass = q.sum(1) + q_rest
    top = z.amax(1)
    state = torch.stack((top, total - top / T, rest_max,
                         torch.where(there, rest_total - rest_max / T, 0.0),
                         torch.where(there, mass * p_rest - q_rest, 0.0), t_max, t_log, mass - 1.0),
                        1)
    return {"loss": loss.masked_fill(dead, math.nan),
            "state": state.masked_fill(dead[:, None], math.nan), "status": dead.to(torch.int32)}


def _exact_grad(s, rows):
    y, z, T, teacher, known = _exact_rows(s, rows)
    m, ls, rm, rls, rest, tm, tls, over = (c[:, None] for c in s["state"][rows].double().unbind(1))
    Tc = T[:, None]
    p = ((z - m) / Tc - ls).exp()
    q = teacher.exp() if s["rest"] else ((teacher - tm) / Tc - tls).exp()
    w = ((z - rm) / Tc - rls).exp()
    out = torch.where(known, (1.0 + over) * p - q, rest * w)
    out *= s["grad_loss"][rows].double()[:, None] / Tc
    out[s["status"][rows] != ROW_OK] = 0.0
    return {"grad_logits": out}


def _exact_adapted(s, b):
    z, a = s["logits"][b].double(), int(s["index"][b])
    if a < 0:
        return z
    u = s["down"][a].double() @ s["hidden"][b].double()
    by = 1.0 if s["scale"] is None else float(s["scale"][a])
    return z + by * (s["up"][a].double() @ u)
