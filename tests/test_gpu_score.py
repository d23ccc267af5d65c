"""qs_token_logprobs and qs_token_logprobs_backward (through the binding) against
the oracle in fp64.

Tolerances, with u = 2^-24 (half a float32 step) and a_i = (z_i - m) / T:
- a_i is a difference, a product with a rounded 1 / T (or a quotient) and the
  rounding of both: at most 4 u |a_i|. A weight exp a_i then carries
  4 u |a_i| + 4 u relative (the exponential itself good to two units).
- S is a sum of positive terms along at most `depth` additions: relative
  depth u + 4 u sum p|a| + 4 u. log S adds 2 u |log S| + 4 u.
- log p_t = a_t - log S: 4 u |a_t| + error of log S + u |log p_t|.
- H = log S + sum p|a|, both terms positive: error of log S, plus
  (2 depth + 16) u sum p|a| + 4 u sum p a^2 for the second.
- a gradient element: p (..) with p's relative error 4 u |a| + 8 u (the row
  statistics are inputs), the G slot gradients summed in order, one final
  rounding of half a step of the output type.
"""

import math

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def depth(V):
    """Additions on a term's way into S: at most 64 in a lane's block, then the
    blocks of a lane, the lanes, the waves and the parts of a row."""
    return 128 + V / 2 ** 14


@pytest.fixture(scope="module")
def qs():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import top_sampling_vocabs_amd as qs
    qs.load()
    return qs


def bf16(x):
    """float32 values rounded to bf16 by truncation (exact in both types)."""
    return (np.asarray(x, np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32)


def pack(legal):
    B, V = legal.shape
    W = -(-V // 32)
    bits = np.zeros((B, W * 32), np.uint8)
    bits[:, :V] = legal
    return np.packbits(bits, axis=1, bitorder="little").view(np.uint32).view(np.int32)


def on_gpu(z, dtype, extra=0):
    """[B, V] on the GPU in padded rows (extra: more padding, filled with a value
    that would win every row)."""
    import torch
    B, V = z.shape
    step = 4 if dtype == "f32" else 8
    buf = np.full((B, (-(-V // step) + extra) * step), 3e38, np.float32)
    buf[:, :V] = z
    t = torch.from_numpy(buf).cuda()
    if dtype == "bf16":
        t = t.to(torch.bfloat16)
    return t[:, :V]


def make(seed, B, V, kind):
    rng = np.random.default_rng(seed)
    if kind == "normal":
        z = rng.normal(0, 3, (B, V))
    elif kind == "ties":
        z = rng.integers(-2, 3, (B, V)).astype(float)
    elif kind == "equal":
        z = np.full((B, V), -7.25)
    elif kind == "falling":
        z = np.broadcast_to(-np.arange(V) * (40.0 / V), (B, V)).copy()
    elif kind == "rising":
        z = np.broadcast_to(np.arange(V) * (40.0 / V), (B, V)).copy()
    elif kind == "stripe":
        # the largest tokens all belong to one lane's places
        z = rng.normal(0, 1, (B, V))
        z[:, np.arange(V) % 512 < 8] += 50.0
    elif kind == "wide":
        z = rng.normal(0, 1, (B, V)) * 10.0 ** rng.integers(-3, 5, (B, V))
    elif kind == "negative":
        z = -np.abs(rng.normal(0, 3, (B, V))) - 1e4
    elif kind == "zeros":
        z = np.where(rng.random((B, V)) < 0.5, 0.0, -0.0)
    else:
        raise ValueError(kind)
    return bf16(z)


def tokens_for(rng, B, V, G, pad=True):
    t = rng.integers(0, V, (B, G)).astype(np.int32)
    if pad:
        t[rng.random((B, G)) < 0.15] = -1
    return t


def run(qs, z, dtype, tokens, T=None, legal=None, top_n=0, extra=0, workspace=None):
    import torch
    lg = on_gpu(z, dtype, extra)
    d = dict(temperature=None if T is None else torch.from_numpy(T).cuda(),
             bitmask=None if legal is None else torch.from_numpy(pack(legal)).cuda())
    tok = torch.from_numpy(tokens).cuda()
    out = qs.token_logprobs(lg, tok, entropy=True, top_n=top_n, workspace=workspace, **d)
    torch.cuda.synchronize()
    return lg, tok, d, out


def check_forward(z, tokens, T, legal, top_n, out):
    B, V = z.shape
    o = {k: v.cpu().numpy().astype(np.float64) for k, v in out.items()}
    lps = o["logprobs"].reshape(B, -1)
    for r in range(B):
        w = oracle.score_row(z[r], None if legal is None else legal[r],
                             1.0 if T is None else T[r], tokens[r], top_n)
        assert o["status"][r] == w["status"], (r, o["status"][r], w["status"])
        if w["status"] != oracle.ROW_OK:
            assert np.array_equal(lps[r], w["logprobs"], equal_nan=True), r
            for k in ("row_max", "log_sum", "entropy"):
                assert np.isnan(o[k][r]), (r, k)
        else:
            fin = w["p"] > 0
            X = (w["p"][fin] * -w["a"][fin]).sum()
            X2 = (w["p"][fin] * w["a"][fin] ** 2).sum()
            t_S = U * (depth(V) + 4 * X + 2 * abs(w["log_sum"]) + 8)
            t_H = t_S + U * ((2 * depth(V) + 16) * X + 4 * X2 + 2 * w["entropy"])
            assert o["row_max"][r] == w["row_max"], r
            assert abs(o["log_sum"][r] - w["log_sum"]) <= t_S, (r, o["log_sum"][r], w["log_sum"])
            assert abs(o["entropy"][r] - w["entropy"]) <= t_H, (r, o["entropy"][r], w["entropy"])
            for got, want in [(lps[r], w["logprobs"])] + (
                    [(o["top_logprobs"][r], w["top_logprobs"])] if top_n else []):
                # what lies below the least float32 is -inf in the output's type
                want = np.where(want < np.finfo(np.float32).min, -np.inf, want)
                fin = np.isfinite(want)
                assert np.array_equal(got[~fin], want[~fin]), (r, got, want)
                tol = t_S + U * (4 * np.abs(want[fin] + w["log_sum"]) + np.abs(want[fin]))
                assert (np.abs(got[fin] - want[fin]) <= tol).all(), (r, got, want)
            empty = tokens[r] == -1
            assert (lps[r][empty] == 0).all(), r
        if top_n:
            assert np.array_equal(o["top_ids"][r], w["top_ids"]), \
                (r, o["top_ids"][r][:8], w["top_ids"][:8])
            gone = w["top_ids"] < 0
            assert (o["top_logprobs"][r][gone] == -np.inf).all(), r


SIZES = [1, 2, 7, 8, 9, 63, 64, 65, 511, 512, 513, 1000, 2047, 2049, 5003, 8193, 16384, 16385,
         40003, 131080, 300007]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", SIZES)
def test_sizes(qs, V, dtype):
    """Every length class, with mask, temperatures, padded slots, top tokens."""
    rng = np.random.default_rng(V)
    B = 5
    z = make(V, B, V, "normal")
    legal = rng.random((B, V)) < 0.4
    legal[0] = True
    legal[3] = False                       # a row without a legal token
    legal[4] = False
    legal[4, V // 2] = True                # and one with a single one
    z[~legal] = np.array([np.nan, np.inf, 3e38, -np.inf], np.float32)[
        rng.integers(0, 4, (~legal).sum())]
    T = rng.uniform(0.3, 2.0, B).astype(np.float32)
    tokens = tokens_for(rng, B, V, 3)
    top_n = int(rng.choice([0, 1, 5, 20, 64]))
    print(f"score V={V} {dtype} top_n={top_n}", flush=True)
    for n in sorted({0, top_n, 64}):
        _, _, _, out = run(qs, z, dtype, tokens, T, legal, n, extra=1)
        check_forward(z, tokens, T, legal, n, out)
    free = make(V + 1, B, V, "normal")
    _, _, _, out = run(qs, free, dtype, tokens, None, None, 7)
    check_forward(free, tokens, None, None, 7, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["ties", "equal", "falling", "rising", "stripe", "wide",
                                  "negative", "zeros"])
@pytest.mark.parametrize("V", [700, 9001, 70000])
def test_values(qs, V, kind, dtype):
    """Ties, ordered rows, one lane's places on top, wide ranges, all negative."""
    print(f"score values V={V} {kind} {dtype}", flush=True)
    B = 3
    z = make(V, B, V, kind)
    tokens = tokens_for(np.random.default_rng(V), B, V, 2, pad=False)
    for n in (1, 20, 64):
        _, _, _, out = run(qs, z, dtype, tokens, None, None, n)
        check_forward(z, tokens, None, None, n, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 40, 3001, 50000])
def test_row_errors(qs, V, dtype):
    """Every row error beside rows that are fine, and values that are legal."""
    print(f"score errors V={V} {dtype}", flush=True)
    rng = np.random.default_rng(V)
    B = 16
    z = make(5, B, V, "normal")
    T = np.ones(B, np.float32)
    legal = np.ones((B, V), bool)
    tokens = tokens_for(rng, B, V, 4)
    z[0, V - 1] = np.nan
    z[1, 0] = np.inf
    z[2, :] = -np.inf
    z[3, :] = -np.inf
    z[3, V // 2] = np.nan                  # NaN among -inf
    legal[4] = False
    z[5, V - 1] = np.nan
    legal[5, V - 1] = V == 1               # NaN at an illegal place
    T[6], T[7], T[8], T[9] = 0.0, -1.0, np.nan, np.inf
    tokens[10, 0] = V
    tokens[11, 3] = -2
    z[12, : V // 2] = -np.inf              # legal -inf tokens
    T[13] = 1e-38
    T[14] = 3e38
    tokens[15] = -1
    _, _, _, out = run(qs, z, dtype, tokens, T, legal, 9)
    check_forward(z, tokens, T, legal, 9, out)


@pytest.mark.parametrize("G", [1, 2, 63, 300, 1024])
def test_many_tokens(qs, G):
    """Many given tokens of a row, repeats among them."""
    print(f"score G={G}", flush=True)
    rng = np.random.default_rng(G)
    z = make(G, 4, 6007, "normal")
    tokens = tokens_for(rng, 4, 6007, G)
    tokens[1] = tokens[1, 0]
    _, _, _, out = run(qs, z, "bf16", tokens, None, None, 0)
    check_forward(z, tokens, None, None, 0, out)


@pytest.mark.parametrize("B,V", [(1, 151936), (2, 600), (300, 2000), (1500, 777)])
def test_batches(qs, B, V):
    """From one long row (spread over the GPU) to more rows than compute units;
    the same call twice gives the same bits."""
    import torch
    print(f"score batch B={B} V={V}", flush=True)
    z = make(B, B, V, "normal")
    tokens = tokens_for(np.random.default_rng(B), B, V, 1)
    for dtype in ("f32", "bf16"):
        _, _, _, out = run(qs, z, dtype, tokens, None, None, 20)
        check_forward(z, tokens, None, None, 20, out)
        _, _, _, again = run(qs, z, dtype, tokens, None, None, 20)
        for k in out:
            assert torch.equal(out[k].view(torch.int32), again[k].view(torch.int32)), k


# --------------------------------------------------------------------------

def check_grad(z, dtype, tokens, T, legal, gl, gH, out, grad):
    B, V = z.shape
    got = grad.float().cpu().numpy().astype(np.float64)
    st = {k: v.cpu().numpy() for k, v in out.items()}
    half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    for r in range(B):
        if st["status"][r] != oracle.ROW_OK:
            assert (got[r] == 0).all(), r
            continue
        Tr = 1.0 if T is None else float(T[r])
        lg = None if legal is None else legal[r]
        H = st["entropy"][r]
        want = oracle.grad_row(z[r], lg, Tr, tokens[r], gl[r], None if gH is None else gH[r],
                               st["row_max"][r], st["log_sum"][r], H)
        ok = np.ones(V, bool) if lg is None else lg
        assert (got[r][~ok] == 0).all(), r
        with np.errstate(over="ignore", invalid="ignore"):
            a = np.where(ok, (z[r].astype(np.float64) - st["row_max"][r]) / Tr, 0.0)
        a = np.maximum(a, -1e4)
        lp = a - st["log_sum"][r]
        p = np.exp(lp)
        live = tokens[r] >= 0
        g_abs = np.abs(gl[r][live]).sum()
        gh = 0.0 if gH is None else abs(float(gH[r]))
        slot = np.zeros(V)
        for t, g in zip(tokens[r][live], gl[r][live]):
            slot[t] += abs(g)
        n = len(tokens[r])
        tol = U / Tr * (p * ((4 * np.abs(a) + 24 + n) * (g_abs + gh * (np.abs(lp) + abs(H)))
                             + gh * 8 * np.abs(a)) + (n + 4) * slot)
        # a p below the least normal float32, 2^-126, may be taken as 0, and so may
        # an element below it: off by 2^-126 times p's factor, and by 2^-126
        tol = tol + 2.0 ** -126 * (1 + (g_abs + gh * (np.abs(lp) + abs(H))) / Tr)
        tol = tol * 1.01 + half * np.abs(want) * 1.01
        bad = np.abs(got[r] - want) > tol
        assert not bad.any(), (r, np.nonzero(bad)[0][:4], got[r][bad][:4], want[bad][:4])


def run_grad(qs, z, dtype, tokens, T, legal, gl, gH, extra=0, **kw):
    import torch
    lg, tok, d, out = run(qs, z, dtype, tokens, T, legal, extra=extra)
    ent = {} if gH is None else dict(entropy=out["entropy"], grad_entropy=torch.from_numpy(gH).cuda())
    grad = qs.token_logprobs_backward(lg, tok, out["row_max"], out["log_sum"], out["status"],
                                      torch.from_numpy(gl).cuda(), **d, **ent, **kw)
    torch.cuda.synchronize()
    return lg, out, grad


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", SIZES)
def test_grad_sizes(qs, V, dtype):
    print(f"grad V={V} {dtype}", flush=True)
    rng = np.random.default_rng(V)
    B = 5
    z = make(V, B, V, "normal")
    legal = rng.random((B, V)) < 0.4
    legal[0] = True
    legal[3] = False
    z[~legal] = np.array([np.nan, np.inf, 3e38, -np.inf], np.float32)[
        rng.integers(0, 4, (~legal).sum())]
    z[1, legal[1]] = np.where(rng.random(legal[1].sum()) < 0.3, -np.inf, z[1, legal[1]])
    T = rng.uniform(0.3, 2.0, B).astype(np.float32)
    tokens = tokens_for(rng, B, V, 3)
    tokens[2, 1:] = tokens[2, 0]           # one token in several slots
    gl = rng.normal(0, 1, (B, 3)).astype(np.float32)
    gl[tokens == -1] = np.nan              # what an empty slot holds is not read into sums
    gH = rng.normal(0, 0.1, B).astype(np.float32)
    _, out, grad = run_grad(qs, z, dtype, tokens, T, legal, gl, gH, extra=1)
    check_grad(z, dtype, tokens, T, legal, gl, gH, out, grad)
    z = make(V + 1, B, V, "normal")
    gl = rng.normal(0, 1, (B, 1)).astype(np.float32)
    t1 = tokens_for(rng, B, V, 1, pad=False)
    _, out, grad = run_grad(qs, z, dtype, t1, None, None, gl, None)
    check_grad(z, dtype, t1, None, None, gl, None, out, grad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G", [1, 2, 9, 300, 1024])
def test_grad_many_tokens(qs, G, dtype):
    print(f"grad G={G} {dtype}", flush=True)
    rng = np.random.default_rng(G)
    B, V = 4, 9007
    z = make(G, B, V, "wide")
    tokens = tokens_for(rng, B, V, G)
    tokens[1] = V - 1
    tokens[2] = np.arange(G) % 17
    gl = rng.normal(0, 1, (B, G)).astype(np.float32)
    gH = rng.normal(0, 1, B).astype(np.float32)
    _, out, grad = run_grad(qs, z, dtype, tokens, None, None, gl, gH)
    check_grad(z, dtype, tokens, None, None, gl, gH, out, grad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grad_in_place_and_padding(qs, dtype):
    """In the logits' own buffer, and into a buffer whose padding stays."""
    import torch
    print(f"grad in place {dtype}", flush=True)
    rng = np.random.default_rng(3)
    B, V = 7, 5003
    z = make(3, B, V, "normal")
    tokens = tokens_for(rng, B, V, 2)
    gl = rng.normal(0, 1, (B, 2)).astype(np.float32)
    _, out, want = run_grad(qs, z, dtype, tokens, None, None, gl, None)
    lg, tok, d, _ = run(qs, z, dtype, tokens)
    got = qs.token_logprobs_backward(lg, tok, out["row_max"], out["log_sum"], out["status"],
                                     torch.from_numpy(gl).cuda(), out=lg)
    torch.cuda.synchronize()
    assert got.data_ptr() == lg.data_ptr() and torch.equal(got, want)
    buf = torch.full((B, V + 61), 7.0, dtype=want.dtype, device="cuda")
    lg = on_gpu(z, dtype)
    qs.token_logprobs_backward(lg, tok, out["row_max"], out["log_sum"], out["status"],
                               torch.from_numpy(gl).cuda(), out=buf[:, :V])
    torch.cuda.synchronize()
    assert torch.equal(buf[:, :V], want) and (buf[:, V:] == 7.0).all()


def test_gradient_against_differences(qs):
    """Central differences of the forward kernel's own outputs. With step h the
    difference carries 2 t / (2 h) of the forward's error t and h^2 / 6 of the
    third derivative (at most 1 in size for log-probabilities, and below 4 for
    the entropy of 12 tokens, where |ln p| < 8)."""
    import torch
    rng = np.random.default_rng(11)
    V, h = 12, 2.0 ** -5
    z = rng.normal(0, 1, V).astype(np.float32)
    z = np.round(z * 256) / 256            # z + h is exact
    T = np.float32(1.25)
    tokens = np.array([3, 7, 3], np.int32)
    gl = np.array([0.7, -1.1, 0.4], np.float32)
    gH = np.float32(0.6)
    rows = np.stack([z] + [z + s * h * np.eye(V, dtype=np.float32)[i]
                           for i in range(V) for s in (1, -1)]).astype(np.float32)
    n = rows.shape[0]
    _, _, _, out = run(qs, rows, "f32", np.tile(tokens, (n, 1)), np.full(n, T, np.float32))
    f = (out["logprobs"].double() * torch.from_numpy(gl).cuda().double()).sum(1) \
        + float(gH) * out["entropy"].double()
    f = f.cpu().numpy()
    want = (f[1::2] - f[2::2]) / (2 * h)
    _, out, grad = run_grad(qs, z[None], "f32", tokens[None], np.array([T]), None, gl[None],
                            np.array([gH]))
    weight = np.abs(gl).sum() + abs(gH)
    tol = weight * (U * 160 * 2 / (2 * h) + 4 * h * h / 6 / float(T) ** 3)
    assert (np.abs(grad[0].cpu().numpy() - want) <= tol).all(), (grad[0].cpu().numpy(), want, tol)


def test_autograd(qs):
    """backward() through the binding: the same gradients, leaves of padded rows,
    outputs without a gradient, one loss of both outputs and of each alone."""
    import torch
    rng = np.random.default_rng(5)
    B, V = 6, 1001
    z = make(5, B, V, "normal")
    tokens = tokens_for(rng, B, V, 2)
    T = rng.uniform(0.5, 1.5, B).astype(np.float32)
    gl = rng.normal(0, 1, (B, 2)).astype(np.float32)
    gH = rng.normal(0, 1, B).astype(np.float32)
    tok, Tt = torch.from_numpy(tokens).cuda(), torch.from_numpy(T).cuda()
    g_l, g_H = torch.from_numpy(gl).cuda(), torch.from_numpy(gH).cuda()
    for dtype in ("f32", "bf16"):
        for use in ("both", "logprobs", "entropy"):
            lg = on_gpu(z, dtype).detach().requires_grad_()
            out = qs.token_logprobs(lg, tok, temperature=Tt, entropy=True, top_n=3)
            assert not out["top_logprobs"].requires_grad and not out["row_max"].requires_grad
            loss = 0
            if use != "entropy":
                loss = loss + (out["logprobs"] * g_l).sum()
            if use != "logprobs":
                loss = loss + (out["entropy"] * g_H).sum()
            (grad,) = torch.autograd.grad(loss, lg)
            torch.cuda.synchronize()
            check_grad(z, dtype, tokens, T, None, gl if use != "entropy" else 0 * gl,
                       gH if use != "logprobs" else None, {k: v.detach() for k, v in out.items()},
                       grad)


def test_autograd_outputs_in_place(qs):
    """The log-probabilities may be changed in place (a masked sum does so). The
    entropy, which the gradient reads, may not: torch reports it."""
    import torch
    z = torch.randn(4, 512, device="cuda")
    tok = torch.tensor([1, 500, -1, 3], dtype=torch.int32, device="cuda")
    keep = (tok >= 0).float()
    grads = []
    for in_place in (False, True):
        lg = z.clone().requires_grad_()
        out = qs.token_logprobs(lg, tok, entropy=True)
        lp, ent = out["logprobs"], out["entropy"]
        if in_place:
            lp *= keep
        else:
            lp = lp * keep
        ent = ent * keep
        (lp.sum() + 0.5 * ent.sum()).backward()
        torch.cuda.synchronize()
        grads.append(lg.grad)
    assert torch.equal(*grads) and bool(grads[0].any())
    with pytest.raises(RuntimeError):
        out = qs.token_logprobs(z.clone().requires_grad_(), tok, entropy=True)
        out["entropy"].mul_(keep)
        out["entropy"].sum().backward()


def test_refusals(qs):
    import torch
    lg = torch.zeros(4, 64, device="cuda")
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    stats = dict(row_max=torch.zeros(4, device="cuda"), log_sum=torch.zeros(4, device="cuda"),
                 status=tok)
    g = torch.zeros(4, device="cuda")
    for kw in (dict(tokens=tok.long()), dict(tokens=tok[:3]), dict(tokens=tok.cpu()),
               dict(tokens=torch.zeros(4, 2, 2, dtype=torch.int32, device="cuda")),
               dict(temperature=torch.ones(3, device="cuda")),
               dict(temperature=torch.ones(4)), dict(logits=lg.half()), dict(logits=lg.cpu()),
               dict(logits=lg.t()), dict(bitmask=torch.zeros(4, 2, device="cuda"))):
        a = dict(logits=lg, tokens=tok) | kw
        with pytest.raises((ValueError, TypeError)):
            qs.token_logprobs(a.pop("logits"), a.pop("tokens"), **a)
    for kw in (dict(top_n=65), dict(top_n=-1), dict(bitmask=torch.zeros(4, 1, dtype=torch.int32,
                                                                        device="cuda"))):
        with pytest.raises(RuntimeError):
            qs.token_logprobs(lg, tok, **kw)
    with pytest.raises(RuntimeError):      # rows that do not start 16-byte aligned
        qs.token_logprobs(torch.zeros(4, 63, device="cuda"), tok)
    with pytest.raises(RuntimeError):      # no token to score
        qs.token_logprobs(lg, torch.zeros(4, 0, dtype=torch.int32, device="cuda"))
    for kw in (dict(grad_logprobs=g[:3]), dict(grad_logprobs=g.double()), dict(entropy=g),
               dict(grad_entropy=g), dict(out=lg.bfloat16()), dict(out=lg[:, :32]),
               dict(out=torch.zeros(4, 64))):
        a = dict(grad_logprobs=g) | kw
        with pytest.raises(ValueError):
            qs.token_logprobs_backward(lg, tok, stats["row_max"], stats["log_sum"],
                                       stats["status"], a.pop("grad_logprobs"), **a)
    out = qs.token_logprobs(lg[:0], tok[:0], entropy=True, top_n=2)
    assert out["logprobs"].shape == (0,) and out["top_ids"].shape == (0, 2)


def test_offsets_past_32_bits(qs):
    """Rows 4 GiB apart, forward and in-place backward: the compact rows' bits."""
    import torch
    print("offsets past 32 bits", flush=True)
    rng = np.random.default_rng(12)
    for V in (5001, 40003):
        z = torch.from_numpy(rng.normal(0, 3, (3, V)).astype(np.float32)).cuda()
        flat = torch.empty((3, -(-V // 8) * 8), device="cuda")[:, :V]
        flat.copy_(z)
        far = torch.empty((3, 1 << 30), device="cuda")[:, :V]
        far.copy_(z)
        tok = torch.from_numpy(rng.integers(0, V, (3, 2)).astype(np.int32)).cuda()
        a = qs.token_logprobs(flat, tok, entropy=True, top_n=5)
        b = qs.token_logprobs(far, tok, entropy=True, top_n=5)
        torch.cuda.synchronize()
        for k in a:
            assert torch.equal(a[k], b[k]), k
        g = torch.ones(3, 2, device="cuda")
        want = qs.token_logprobs_backward(flat, tok, a["row_max"], a["log_sum"], a["status"], g)
        got = qs.token_logprobs_backward(far, tok, b["row_max"], b["log_sum"], b["status"], g,
                                         out=far)
        torch.cuda.synchronize()
        assert torch.equal(want, got)
        del far, got, b


def test_longest_row(qs):
    """2^30 tokens, the most a row may have. All logits are 0 but three, so that
    S = V - 3 + e^1 + e^2 + e^3 before the maximum is taken out. Its terms pass at
    most 64 additions in a lane, 6 + 4 in a workgroup, 2^15 / 64 and 6 in the join:
    log S is off by at most 600 * 2^-24 = 3.6e-5, its own rounding to float32
    (2^-24 * 18) within that."""
    import torch
    print("longest row", flush=True)
    V = 1 << 30
    z = torch.zeros((1, V), dtype=torch.bfloat16, device="cuda")
    at = [V - 1, 12345678, (1 << 29) + 7]
    for k, i in enumerate(at):
        z[0, i] = float(3 - k)
    tok = torch.tensor([[V - 1, 0, at[2], -1]], dtype=torch.int32, device="cuda")
    out = qs.token_logprobs(z, tok, top_n=3)
    torch.cuda.synchronize()
    S = V - 3 + sum(math.exp(k) for k in (1, 2, 3))
    assert out["status"].item() == 0 and out["row_max"].item() == 3.0
    assert abs(out["log_sum"].item() - (math.log(S) - 3)) <= 3.6e-5
    assert out["top_ids"].tolist() == [[V - 1, at[1], at[2]]]
    lp = out["logprobs"][0].tolist()
    for got, zv in zip(lp, (3.0, 0.0, 1.0)):
        assert abs(got - (zv - math.log(S))) <= 3.6e-5 + 2 ** -20
    assert lp[3] == 0.0
    g = torch.ones_like(tok, dtype=torch.float32)
    grad = qs.token_logprobs_backward(z, tok, out["row_max"], out["log_sum"], out["status"], g,
                                      out=z)
    torch.cuda.synchronize()
    # three slots: 1 - 3 p at a given token, -3 p elsewhere, p below 2e-8
    assert grad[0, V - 1].item() == 1.0 and grad[0, at[2]].item() == 1.0
    p = 3 * math.exp(2) / S
    assert abs(grad[0, at[1]].item() + p) <= p * 2 ** -7


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 1000, 32003, 151937])
def test_peaked_rows(qs, V, dtype):
    """Rows that one token nearly wins alone keep relative precision: with q the
    mass beside the largest token, log S = -ln(1 - q) has the relative error of
    the sum of the other weights, U (depth + 8) q + 4 U X as in check_forward
    with the one left out, and that of log1p (2 steps)."""
    import torch
    print(f"peaked V={V} {dtype}", flush=True)
    rng = np.random.default_rng(V)
    up = np.array([12.0, 16.0, 20.0, 26.0, 34.0])
    z = rng.normal(0, 2, (5, V))
    at = rng.integers(0, V, 5)
    z[np.arange(5), at] = up
    z = bf16(z)
    tokens = np.stack((at, (at + 1) % V), 1).astype(np.int32)
    T = np.array([1.0, 1.0, 0.7, 1.3, 1.0], np.float32)
    _, _, _, out = run(qs, z, dtype, tokens, T=T, top_n=1)
    o = {k: v.cpu().numpy().astype(np.float64) for k, v in out.items()}
    for r in range(5):
        w = oracle.score_row(z[r], None, T[r], tokens[r], 1)
        fin = w["p"] > 0
        X = (w["p"][fin] * -w["a"][fin]).sum()
        X2 = (w["p"][fin] * w["a"][fin] ** 2).sum()
        rest = np.delete(w["p"], at[r]).sum()
        logS = np.log1p(rest / (1 - rest)) if rest < 0.5 else w["log_sum"]
        tol = U * ((depth(V) + 8) * rest + 4 * X + 4 * logS) + 1e-37
        assert abs(o["log_sum"][r] - logS) <= tol, (r, o["log_sum"][r], logS)
        assert abs(o["logprobs"][r][0] + logS) <= tol
        assert o["top_logprobs"][r][0] == o["logprobs"][r][0]
        H = logS + X
        t_H = tol + U * ((2 * depth(V) + 16) * X + 4 * X2 + 2 * H) + 1e-37
        assert abs(o["entropy"][r] - H) <= t_H, (r, o["entropy"][r], H)


def gap_rows(seed, B, V):
    """Rows with a stretch of V / 3 tokens (whole waves and parts of long rows) that
    is illegal in the rows 1, 4, .. and legal but -inf in the rows 2, 5, .."""
    z = make(seed, B, V, "normal")
    legal = np.random.default_rng(seed).random((B, V)) < 0.6
    legal[:, V - 1] = True
    gap = slice(V // 3, 2 * V // 3)
    legal[1::3, gap] = False
    z[2::3, gap] = -np.inf
    return z, legal


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 40, 700, 3001, 100003])
def test_temperatures(qs, V, dtype):
    """Every power of ten that a temperature can be, beside waves and parts
    without a legal or a finite token."""
    print(f"score temperatures V={V} {dtype}", flush=True)
    T = np.repeat(10.0 ** np.arange(-37, 39), 3).astype(np.float32)
    B = T.size
    z, legal = gap_rows(V, B, V)
    tokens = tokens_for(np.random.default_rng(V), B, V, 2)
    for n in (0, 5):
        _, _, _, out = run(qs, z, dtype, tokens, T, legal, n)
        check_forward(z, tokens, T, legal, n, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 3001, 100003])
def test_large_logits(qs, V, dtype):
    """Logits up to 1e37 as they are and at temperatures of their own size, and
    (float32) whole numbers beside a large offset, where neighbours differ by 1."""
    print(f"score large logits V={V} {dtype}", flush=True)
    e = np.repeat(np.arange(0, 37), 2)
    B = e.size
    z, legal = gap_rows(V, B, V)
    z = bf16(z * (10.0 ** e)[:, None])
    T = np.where(np.arange(B) % 2 == 0, 1.0, 10.0 ** e).astype(np.float32)
    tokens = tokens_for(np.random.default_rng(V), B, V, 2)
    _, _, _, out = run(qs, z, dtype, tokens, T, legal, 3)
    check_forward(z, tokens, T, legal, 3, out)
    if dtype == "f32":
        rng = np.random.default_rng(V + 1)
        base = np.repeat(2.0 ** np.array([8, 16, 20, 22, 23, -8, -16, -20, -22, -23]), 4)
        base = np.where(np.arange(base.size) // 4 < 5, base, -(base ** -1.0))
        z = (base[:, None] + rng.integers(0, 40, (base.size, V))).astype(np.float32)
        T = np.tile([4.0, 1.0, 0.25, 0.01], base.size // 4).astype(np.float32)
        tokens = tokens_for(rng, base.size, V, 2)
        _, _, _, out = run(qs, z, "f32", tokens, T, None, 3)
        check_forward(z, tokens, T, None, 3, out)


@pytest.mark.parametrize("dtype,V", [("f32", 32769), ("f32", 40003), ("bf16", 131077)])
def test_caller_workspace(qs, V, dtype):
    """Rows of several parts with the caller's scratch memory, used again for
    smaller and other calls: the bits of a call that makes its own. What cannot
    hold the call is refused."""
    import torch
    print(f"score workspace V={V} {dtype}", flush=True)
    B = 6
    z = make(V, B, V, "normal")
    tokens = tokens_for(np.random.default_rng(V), B, V, 2)
    _, _, _, want = run(qs, z, dtype, tokens, None, None, 20)
    check_forward(z, tokens, None, None, 20, want)
    lg = on_gpu(z, dtype)
    tok = torch.from_numpy(tokens).cuda()
    ws = qs.token_logprobs_workspace_for(lg, 20)
    assert ws is not None and ws.device == lg.device
    for fill in (0, 255):
        ws.fill_(fill)
        got = qs.token_logprobs(lg, tok, entropy=True, top_n=20, workspace=ws)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got[k].view(torch.int32), want[k].view(torch.int32)), k
    small = qs.token_logprobs(lg[:2], tok[:2], entropy=True, workspace=ws)
    leaf = lg.detach().requires_grad_()
    out = qs.token_logprobs(leaf, tok, workspace=ws)
    (grad,) = torch.autograd.grad(out["logprobs"].sum(), leaf)
    torch.cuda.synchronize()
    assert torch.equal(small["logprobs"], want["logprobs"][:2])
    assert torch.equal(out["logprobs"], want["logprobs"]) and bool(torch.isfinite(grad).all())
    n = ws.numel()
    for bad in (ws.cpu(), ws[:1].expand(n), torch.empty(2 * n, dtype=torch.uint8,
                                                        device="cuda")[::2]):
        with pytest.raises(ValueError):
            qs.token_logprobs(lg, tok, top_n=20, workspace=bad)
    for bad in (ws[:n - 1], ws[256:], torch.empty(n + 64, dtype=torch.uint8, device="cuda")[64:]):
        with pytest.raises(RuntimeError):
            qs.token_logprobs(lg, tok, top_n=20, workspace=bad)


@pytest.mark.parametrize("G", [1, 3])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grad_of_non_finite_gradients(qs, dtype, G):
    """A NaN or an infinity in an incoming gradient reaches every legal token of its
    row, whatever token it belongs to, and no other row. Illegal tokens and rows
    with an error stay 0."""
    import torch
    print(f"grad non-finite {dtype} G={G}", flush=True)
    rng = np.random.default_rng(21)
    V, bad = 5003, [np.nan, np.inf, -np.inf]
    B = 16
    z = make(21, B, V, "normal")
    legal = rng.random((B, V)) < 0.5
    legal[:, 0], legal[:, 1] = True, False
    legal[12] = False                      # a row without a legal token
    tokens = rng.integers(2, V, (B, G)).astype(np.int32)
    gl = rng.normal(0, 1, (B, G)).astype(np.float32)
    gH = rng.normal(0, 1, B).astype(np.float32)
    for r in range(3):
        tokens[r, -1], gl[r, -1] = 0, bad[r]          # a legal token's gradient
        tokens[3 + r, -1], gl[3 + r, -1] = 1, bad[r]  # an illegal one's
        gH[6 + r] = bad[r]
    gl[9, 0], gH[9] = np.inf, -np.inf
    gl[12], gH[12] = np.nan, np.nan
    tokens[13, 0], gl[13, 0] = -1, np.nan             # an empty slot's is not read
    for use_entropy in (True, False):
        g = gH if use_entropy else None
        _, out, grad = run_grad(qs, z, dtype, tokens, None, legal, gl, g)
        got = grad.float().cpu().numpy()
        lost = [r for r in range(10) if use_entropy or not 6 <= r < 9]
        for r in range(B):
            if r in lost:
                assert not np.isfinite(got[r][legal[r]]).any(), r
                if r in (0, 3, 6):
                    assert np.isnan(got[r][legal[r]]).all(), r
                assert (got[r][~legal[r]] == 0).all(), r
        keep = [r for r in range(B) if r not in lost]
        pick = {k: v[keep] for k, v in out.items()}
        check_grad(z[keep], dtype, tokens[keep], None, legal[keep], gl[keep],
                   None if g is None else g[keep], pick, grad[keep])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grad_past_the_largest_value(qs, dtype):
    """Finite gradients whose quotient by T overflows: a token without weight still
    gets 0 (not 0 times an infinity), and the row holds no NaN."""
    import torch
    z = np.full((2, 600), -1e4, np.float32)
    z[:, 7] = 0.0
    z[0, 8] = 0.0
    tokens = np.array([[7], [9]], np.int32)
    T = np.array([1e-9, 1e-9], np.float32)
    gl = np.full((2, 1), 1e35, np.float32)
    gH = np.full(2, 1e35, np.float32)
    _, out, grad = run_grad(qs, z, dtype, tokens, T, None, gl, gH)
    got = grad.float().cpu().numpy()
    assert not np.isnan(got).any()
    still = np.ones(600, bool)
    still[[7, 8, 9]] = False
    assert (got[:, still] == 0).all() and got[0, 7] > 1e38 and got[0, 8] < -1e38


def test_writes_are_seen_by_autograd(qs):
    """A buffer that a call writes into counts as changed: a graph that saved it
    reports so, as for torch's own writes. Leaves that require a gradient are
    refused as outputs; tensors of inference mode are taken."""
    import torch
    torch.manual_seed(1)
    B, V, K = 4, 512, 256
    hidden = torch.randn(B, K, device="cuda").bfloat16()
    codes = torch.randint(0, 256, (V, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.rand(V, K // 64, device="cuda") * 0.02
    tok = torch.randint(0, V, (B,), dtype=torch.int32, device="cuda")
    T, k, p = (torch.full((B,), v, device="cuda") for v in (1.0, 0, 1.0))
    sample = (codes, scales, None, T, k.int(), p)
    buf = torch.empty(B, V, device="cuda")
    base = qs.token_logprobs(qs.head_logits(hidden, codes, scales, out=buf), tok)
    grad_args = (tok, base["row_max"], base["log_sum"], base["status"],
                 torch.ones(B, device="cuda"))
    history = torch.zeros(B, 3, dtype=torch.int32, device="cuda")
    count, one = torch.full((B,), 3, dtype=torch.int32, device="cuda"), torch.ones(B, device="cuda")
    writes = {
        "head_logits": lambda t: qs.head_logits(hidden, codes, scales, out=t),
        "sample_hidden": lambda t: qs.sample_hidden(hidden, *sample, logits=t,
                                                    uniforms=torch.zeros(B, dtype=torch.float64,
                                                                         device="cuda")),
        "backward": lambda t: qs.token_logprobs_backward(buf, *grad_args, out=t),
        "penalties": lambda t: qs.apply_penalties(t, history, count, 2 * one, one),
        "bias": lambda t: qs.apply_logit_bias(t, history, torch.ones(B, 3, device="cuda"), count),
    }
    for name, write in writes.items():
        z = torch.randn(B, V, device="cuda").requires_grad_()
        kept = z.detach()                  # shares its memory and its version
        before = kept._version
        out = qs.token_logprobs(z, tok)
        write(kept)
        assert kept._version > before, name
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out["logprobs"].sum().backward()
        with torch.inference_mode():
            write(torch.zeros(B, V, device="cuda"))
    for name in ("head_logits", "sample_hidden", "backward"):
        leaf = torch.zeros(B, V, device="cuda").requires_grad_()
        for t in (leaf, leaf * 2):
            with pytest.raises(ValueError, match="gradient"):
                writes[name](t)
        with torch.no_grad():
            writes[name](leaf)
    torch.cuda.synchronize()


def test_forward_mode_is_refused(qs):
    """Tangents are not carried: a dual tensor is refused, not taken without its
    tangent. Under a dual level plain tensors work as ever."""
    import torch
    from torch.autograd import forward_ad
    torch.manual_seed(2)
    B, V, K = 3, 512, 128
    z = torch.randn(B, V, device="cuda")
    tok = torch.randint(0, V, (B,), dtype=torch.int32, device="cuda")
    T = torch.ones(B, device="cuda")
    hidden = torch.randn(B, K, device="cuda").bfloat16()
    codes = torch.randint(0, 256, (V, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.rand(V, K // 64, device="cuda")
    out = qs.token_logprobs(z, tok, entropy=True)
    stats = (out["row_max"], out["log_sum"], out["status"])
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t, torch.ones_like(t))
        again = qs.token_logprobs(z, tok, entropy=True)
        qs.head_logits(hidden, codes, scales)
        qs.token_logprobs_backward(z, tok, *stats, T)
        for call in (lambda: qs.token_logprobs(dual(z), tok),
                     lambda: qs.token_logprobs(dual(z.clone().requires_grad_()), tok),
                     lambda: qs.token_logprobs(z, tok, temperature=dual(T)),
                     lambda: qs.token_logprobs_backward(dual(z), tok, *stats, T),
                     lambda: qs.token_logprobs_backward(z, tok, *stats, dual(T)),
                     lambda: qs.token_logprobs_backward(z, tok, *stats, T, entropy=out["entropy"],
                                                        grad_entropy=dual(T)),
                     lambda: qs.head_logits(dual(hidden), codes, scales),
                     lambda: qs.head_logits(hidden, codes, dual(scales))):
            with pytest.raises(ValueError, match="forward"):
                call()
    torch.cuda.synchronize()
    assert torch.equal(again["logprobs"], out["logprobs"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 1000, 32003])
def test_grad_of_peaked_rows(qs, V, dtype):
    """The gradient at a token that is almost certain keeps relative precision.
    With lp = -log S there (a = 0, so log S alone rounds nothing) its own slots give
    -g expm1(lp): a rounding each of the sum of the slots, of expm1 (two units),
    of the product and of the quotient; the other slots' sum times p, with p's few
    units; and p (lp + H) gH, both terms of one size."""
    import torch
    print(f"grad peaked V={V} {dtype}", flush=True)
    rng = np.random.default_rng(V)
    B = 8
    z = rng.normal(0, 2, (B, V))
    at = rng.integers(0, V, B)
    z[np.arange(B), at] = [12, 16, 20, 26, 34, 20, 26, 50]
    z = bf16(z)
    T = np.array([1, 1, 0.7, 1.3, 1, 1, 1, 1], np.float32)
    half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    for G in (1, 3):
        tokens = np.repeat(at[:, None], G, 1).astype(np.int32)
        gl = rng.normal(0, 1, (B, G)).astype(np.float32)
        if G == 3:
            tokens[4:, 1] = (at[4:] + 1) % V
            gl[4:, 1] *= 1e-9              # of the size of what the peak leaves
        for gH in (None, rng.normal(0, 1, B).astype(np.float32)):
            _, out, grad = run_grad(qs, z, dtype, tokens, T, None, gl, gH)
            got = grad.float().cpu().numpy().astype(np.float64)
            for r in range(B):
                ls, H = (float(out[k][r]) for k in ("log_sum", "entropy"))
                own = tokens[r] == at[r]
                hit, rest = (gl[r][m].astype(np.float64) for m in (own, ~own))
                p = math.exp(-ls)
                g = 0.0 if gH is None else float(gH[r])
                want = (-hit.sum() * math.expm1(-ls) - rest.sum() * p
                        - g * p * (H - ls)) / T[r]
                tol = U * ((G + 8) * np.abs(hit).sum() * -math.expm1(-ls)
                           + (G + 8) * np.abs(rest).sum() * p
                           + 8 * abs(g) * p * (H + ls)) / T[r]
                tol = tol * 1.01 + half * abs(want) * 1.01 + 2.0 ** -126
                assert abs(got[r, at[r]] - want) <= tol, (r, G, got[r, at[r]], want, tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_largest_temperatures(qs, dtype):
    """Temperatures up to float32's largest value over logits of that size: log2(e) / T
    is below the least normal float32 there, still good to 2^-22 of itself, which
    |a| below 3 turns into 12 units at most (the sums' own tolerance has 128)."""
    print(f"score largest temperatures {dtype}", flush=True)
    T = np.array([1e37, 1e38, 1.2e38, 1.3e38, 2e38, 3e38, 3.4e38], np.float32)
    rng = np.random.default_rng(8)
    B = T.size
    for V in (40, 3001, 70003):
        z = bf16(rng.uniform(-1.6e38, 1.6e38, (B, V)))
        tokens = tokens_for(rng, B, V, 3)
        _, _, _, out = run(qs, z, dtype, tokens, T, None, 4)
        check_forward(z, tokens, T, None, 4, out)


def test_grad_at_largest_temperatures(qs):
    """Gradients large enough that their quotients by such temperatures are normal
    numbers."""
    print("grad largest temperatures", flush=True)
    T = np.array([1e37, 1.2e38, 2e38, 3.4e38], np.float32)
    rng = np.random.default_rng(9)
    B, V = T.size, 3001
    z = bf16(rng.uniform(-1.6e38, 1.6e38, (B, V)))
    tokens = tokens_for(rng, B, V, 2)
    gl = (1e20 * rng.normal(0, 1, (B, 2))).astype(np.float32)
    gH = (1e20 * rng.normal(0, 1, B)).astype(np.float32)
    _, out, grad = run_grad(qs, z, "f32", tokens, T, None, gl, gH)
    check_grad(z, "f32", tokens, T, None, gl, gH, out, grad)


@pytest.mark.parametrize("T", [2e-38, 1e-38, 3e-39, 1e-39, 1e-41])
def test_grad_at_smallest_temperatures(qs, T):
    """Two equal maxima share the row, everything else has no weight: the gradient at
    a given one is g / (2 T), at the other -g / (2 T), by a float32 product and
    quotient, also where 1 / T has no float32."""
    print(f"grad smallest temperature {T}", flush=True)
    z = np.full((1, 300), -2.0, np.float32)
    z[0, [11, 200]] = 1.5
    T = np.array([T], np.float32)
    g = np.float32(float(T[0]) * 1e30)
    _, out, grad = run_grad(qs, z, "f32", np.array([[200]], np.int32), T, None,
                            np.array([[g]], np.float32), None)
    got = grad[0].cpu().numpy().astype(np.float64)
    want = float(g) / (2 * float(T[0]))
    assert abs(got[200] - want) <= 16 * U * want and abs(got[11] + want) <= 16 * U * want
    got[[11, 200]] = 0
    assert (got == 0).all()


@pytest.mark.parametrize("dtype,V", [("bf16", 70001), ("f32", 20001), ("f32", 40001)])
def test_many_tokens_of_long_rows(qs, dtype, V):
    """More given tokens than the workgroup that writes them has threads."""
    print(f"score many tokens V={V} {dtype}", flush=True)
    rng = np.random.default_rng(V)
    z = make(V, 3, V, "normal")
    tokens = tokens_for(rng, 3, V, 1024)
    tokens[2, 1023] = V                    # an error in the last slot
    for n in (0, 20):
        _, _, _, out = run(qs, z, dtype, tokens, None, None, n)
        check_forward(z, tokens, None, None, n, out)


@pytest.mark.parametrize("V", [45, 3001, 70001])
def test_bits_past_the_row_are_ignored(qs, V):
    """Legal bits from V on, in the last word and in a wider stride's words."""
    import torch
    print(f"score bits past the row V={V}", flush=True)
    rng = np.random.default_rng(V)
    B = 3
    z = make(V, B, V, "normal")
    legal = rng.random((B, V)) < 0.5
    legal[2] = False                       # no legal token, whatever lies behind
    tokens = tokens_for(rng, B, V, 2)
    gl = rng.normal(0, 1, (B, 2)).astype(np.float32)
    W = -(-V // 32)
    words = np.full((B, W + 3), 0xFFFFFFFF, np.uint32)
    words[:, :W] = pack(legal).view(np.uint32)
    words[:, W - 1] |= np.uint32((0xFFFFFFFF << (V % 32)) & 0xFFFFFFFF)
    bm = torch.from_numpy(words.view(np.int32)).cuda()[:, :W]
    tok = torch.from_numpy(tokens).cuda()
    for dtype in ("f32", "bf16"):
        lg = on_gpu(z, dtype, extra=1)
        out = qs.token_logprobs(lg, tok, bitmask=bm, entropy=True, top_n=5)
        grad = qs.token_logprobs_backward(lg, tok, out["row_max"], out["log_sum"], out["status"],
                                          torch.from_numpy(gl).cuda(), bitmask=bm)
        torch.cuda.synchronize()
        check_forward(z, tokens, None, legal, 5, out)
        check_grad(z, dtype, tokens, None, legal, gl, None, out, grad)


def test_most_rows(qs):
    """The largest batch, 2^22 - 1 rows. Seven terms of S, so log S is off by 16 + 4 sum
    p |a| units at most (|a| < 64, p |a| below 1/e each) and a log-probability by
    4 |a| units more; a gradient element of size at most 1 by 4 + 4 p |a| units
    and a bf16 half step."""
    import torch
    print("score most rows", flush=True)
    B, V = (1 << 22) - 1, 7
    torch.manual_seed(3)
    z = torch.randn(B, 8, device="cuda").mul_(3).bfloat16()[:, :V]
    tok = torch.randint(0, V, (B,), dtype=torch.int32, device="cuda")
    out = qs.token_logprobs(z, tok, top_n=2)
    lp = torch.log_softmax(z.double(), 1)
    at = tok.long()[:, None]
    want = lp.gather(1, at)[:, 0]
    assert bool((out["status"] == 0).all())
    assert bool(((out["logprobs"] - want).abs() <= U * (64 + 5 * want.abs())).all())
    best = torch.sort(z.float(), dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(out["top_ids"], best.int())
    grad = qs.token_logprobs_backward(z, tok, out["row_max"], out["log_sum"], out["status"],
                                      torch.ones(B, device="cuda"))
    want = (-lp.exp()).scatter_add_(1, at, torch.ones_like(at, dtype=torch.float64))
    tol = 2.0 ** -8 * 1.01 * want.abs() + 64 * U
    assert bool(((grad - want).abs() <= tol).all())


def test_empty_batches(qs):
    """No rows: outputs of the right shape, no error, in every call."""
    import torch
    e = dict(device="cuda")
    z, tok = torch.zeros(0, 64, **e), torch.zeros((0, 2), dtype=torch.int32, **e)
    row, st = torch.zeros(0, **e), torch.zeros(0, dtype=torch.int32, **e)
    grad = qs.token_logprobs_backward(z, tok, row, row, st, torch.zeros((0, 2), **e), entropy=row,
                                      grad_entropy=row)
    assert grad.shape == (0, 64)
    leaf = z.clone().requires_grad_()
    out = qs.token_logprobs(leaf, tok, entropy=True)
    (out["logprobs"].sum() + out["entropy"].sum()).backward()
    assert leaf.grad.shape == (0, 64)
    long = torch.zeros(0, 70016, **e)
    assert qs.token_logprobs_workspace_for(long, 5) is None
    assert qs.token_logprobs(long, tok, top_n=5)["top_ids"].shape == (0, 5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 3001, 70001])
def test_lowest_values(qs, V, dtype):
    """The type's lowest value as a mask: in half a row, in all of it, in all but one
    token, with and without other tokens in the same wave."""
    print(f"lowest values V={V} {dtype}", flush=True)
    rng = np.random.default_rng(V)
    low = np.float32(np.finfo(np.float32).min) if dtype == "f32" else \
        np.uint32(0xFF7F0000).view(np.float32)
    B = 5
    z = make(V, B, V, "normal")
    z[0, rng.random(V) < 0.5] = low
    z[1] = low
    z[2, : V // 2] = low
    z[3] = low
    z[3, V - 1] = -3.0
    z[4] = low
    z[4, 0] = -np.inf
    T = np.array([0.3, 0.7, 2.0, 1.0, 1e-3], np.float32)
    tokens = tokens_for(rng, B, V, 2, pad=False)
    gl = rng.normal(0, 1, (B, 2)).astype(np.float32)
    gH = rng.normal(0, 1, B).astype(np.float32)
    _, _, _, out = run(qs, z, dtype, tokens, T, None, 20)
    check_forward(z, tokens, T, None, 20, out)
    _, out, grad = run_grad(qs, z, dtype, tokens, T, None, gl, gH)
    check_grad(z, dtype, tokens, T, None, gl, gH, out, grad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["spread", "close", "one"])
def test_grad_token_lists(qs, kind, dtype):
    """1024 slots spread over a row, next to each other across the border of two
    workgroups, and all of one token; illegal tokens and empty slots among them.
    In place and twice: the same bits."""
    import torch
    print(f"grad token lists {kind} {dtype}", flush=True)
    rng = np.random.default_rng(31)
    B, V, G = 3, 40003, 1024
    z = make(31, B, V, "normal")
    legal = rng.random((B, V)) < 0.7
    tokens = {"spread": rng.integers(0, V, (B, G)),
              "close": 8192 - G // 4 + rng.integers(0, G // 2, (B, G)),
              "one": np.full((B, G), 8191)}[kind].astype(np.int32)
    tokens[rng.random((B, G)) < 0.1] = -1
    legal[:2, 8191] = True
    legal[2, 8191] = False
    gl = rng.normal(0, 1, (B, G)).astype(np.float32)
    gH = rng.normal(0, 1, B).astype(np.float32)
    _, out, grad = run_grad(qs, z, dtype, tokens, None, legal, gl, gH)
    check_grad(z, dtype, tokens, None, legal, gl, gH, out, grad)
    lg, tok, d, _ = run(qs, z, dtype, tokens, None, legal)
    args = (tok, out["row_max"], out["log_sum"], out["status"], torch.from_numpy(gl).cuda())
    ent = dict(entropy=out["entropy"], grad_entropy=torch.from_numpy(gH).cuda())
    for o in (None, lg):
        again = qs.token_logprobs_backward(lg, *args, out=o, **d, **ent)
        torch.cuda.synchronize()
        assert torch.equal(again, grad)
