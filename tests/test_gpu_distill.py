"""qs_distill_loss and qs_distill_loss_backward (through the binding) against the
oracle in fp64.

Tolerances, with u = 2^-24 (half a float32 step), a_i = (z_i - m_R) / T over the tokens
that the teacher does not name, w their softmax, S_R the sum of exp a:
- a_i is a difference, a product with a rounded 1 / T and the rounding of both: at
  most 4 u |a_i|. A weight exp a_i then carries 4 u |a_i| + 4 u relative. S_R is a sum
  of positive terms along at most `depth` additions:
  e_S = u (depth + 4 sum w|a| + 8) relative.
- the named tokens are worked out in float64, from float32 inputs: log S is off by
  p_R e_S, log S_R by e_S, p_R by p_R (1 - p_R) e_S relative to nothing, and the loss,
  Q log S - q_R log S_R and exact terms, by |Q p_R - q_R| e_S. Beside them 2^-46 of
  the magnitudes that are added up in float64 (some 40 roundings and an exponential
  and a logarithm good to 2 steps each), and each output is rounded once to float32.
- a gradient element of the rest is exp(a_i - log S_R) c with c a product and a
  quotient: u (8 |a_i| + 8 |log S_R| + 16) relative; one of a named token is worked
  out in float64; float32 and output rounding: u and half a step of the type.
"""

import numpy as np
import pytest

import oracle
from test_gpu_score import SIZES, bf16, depth, gap_rows, make, on_gpu, pack

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
D = 2.0 ** -46


@pytest.fixture(scope="module")
def qs():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import top_sampling_vocabs_amd as qs
    qs.load()
    return qs


def teacher(rng, z, legal, T, K, rest, pad=True):
    """Lists of up to K distinct tokens of each row: largest ones and any others, in any
    order, some slots empty, some of probability 0."""
    B, V = z.shape
    ids = np.full((B, K), -1, np.int32)
    values = np.full((B, K), np.nan, np.float32)   # what an empty slot holds is not read
    for r in range(B):
        n = min(K, V)
        y = np.where(np.isfinite(z[r]), z[r], 0.0) * 0.7 + rng.normal(0, 1, V)
        best = np.argsort(-y)[: n // 2 + 1]
        others = rng.permutation(V)
        tok = np.concatenate((best, others[~np.isin(others, best)]))[:n]
        slots = rng.permutation(K)[:n]
        v = y[tok]
        if rest:
            t = 1.0 if T is None else max(min(float(T[r]), 1e3), 1e-3)
            x = y / t
            v = x[tok] - (np.log(np.exp(x - x.max()).sum()) + x.max())
        if pad:
            gone = rng.random(n) < 0.15
            tok, slots, v = tok[~gone], slots[~gone], v[~gone]
            v = np.where(rng.random(v.size) < 0.1, -np.inf, v)
        ids[r, slots] = tok
        with np.errstate(over="ignore"):
            values[r, slots] = v
    return ids, values


def args_of(ids, values, T=None, legal=None):
    import torch
    return (torch.from_numpy(ids).cuda(), torch.from_numpy(values).cuda()), dict(
        temperature=None if T is None else torch.from_numpy(T).cuda(),
        bitmask=None if legal is None else torch.from_numpy(pack(legal)).cuda())


def run(qs, z, dtype, ids, values, T=None, legal=None, rest=False, extra=0, workspace=None):
    import torch
    lg = on_gpu(z, dtype, extra)
    t, d = args_of(ids, values, T, legal)
    out = qs.distill_loss(lg, *t, rest=rest, workspace=workspace, **d)
    torch.cuda.synchronize()
    return lg, t, d, out


def check(z, ids, values, T, legal, rest, out):
    B, V = z.shape
    o = {k: v.cpu().numpy().astype(np.float64) for k, v in out.items()}
    for r in range(B):
        w = oracle.distill_row(z[r], None if legal is None else legal[r],
                               1.0 if T is None else T[r], ids[r], values[r], rest)
        assert o["status"][r] == w["status"], (r, o["status"][r], w["status"])
        if w["status"] != oracle.ROW_OK:
            assert np.isnan(o["loss"][r]) and np.isnan(o["state"][r]).all(), r
            continue
        got, want = o["state"][r], w["state"]
        X = (w["w"] * -np.maximum(w["a"], -1e4)).sum() / max(w["w"].sum(), 1.0)
        e_S = U * (depth(V) + 4 * X + 8)
        pr, Q = w["p_rest"], w["mass"]
        # m, m_R and the teacher's largest value are inputs
        for k in (0, 2, 5):
            assert got[k] == want[k], (r, k, got[k], want[k])
        tiny = 2.0 ** -126
        tol = {1: pr * e_S + U * abs(want[1]), 3: e_S + U * abs(want[3]),
               4: Q * pr * (1 - pr) * e_S + U * abs(want[4]) + D * (Q + 1),
               6: (U + D) * abs(want[6]), 7: U * abs(want[7]) + D * (Q + 1)}
        for k, by in tol.items():
            assert abs(got[k] - want[k]) <= 1.01 * by + tiny, (r, k, got[k], want[k], by)
        loss, want = o["loss"][r], w["loss"]
        if abs(want) > np.finfo(np.float32).max:
            assert loss == want or abs(loss) == np.inf or abs(loss) > 3.4e38, (r, loss, want)
            continue
        by = abs(w["state"][4]) * e_S + U * abs(want) + D * w["size"] + tiny
        assert abs(loss - want) <= 1.01 * by, (r, loss, want, by)




@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", SIZES)
def test_sizes(qs, V, dtype, rest):
    """Every length class with mask, temperatures, short lists, any place of the list's
    tokens; masked places hold NaN, infinities and the largest value."""
    print(f"distill V={V} {dtype} rest={rest}", flush=True)
    rng = np.random.default_rng(V)
    B = 6
    z = make(V, B, V, "normal")
    legal = rng.random((B, V)) < 0.4
    legal[0] = True
    legal[3] = False                       # a row without a legal token
    legal[4] = False
    legal[4, V // 2] = True                # and one with a single one
    z[~legal] = np.array([np.nan, np.inf, 3e38, -np.inf], np.float32)[
        rng.integers(0, 4, (~legal).sum())]
    some = legal[1] & (rng.random(V) < 0.3)
    z[1, some] = -np.inf if not some.all() else z[1, some]
    T = rng.uniform(0.3, 2.0, B).astype(np.float32)
    for K in (1, 5, 70):
        ids, values = teacher(rng, z, legal, T, K, rest)
        ids[5], values[5] = -1, np.nan     # a row without a teacher
        _, _, _, out = run(qs, z, dtype, ids, values, T, legal, rest, extra=1)
        check(z, ids, values, T, legal, rest, out)
    free = make(V + 1, B, V, "normal")
    ids, values = teacher(rng, free, None, None, 20, rest, pad=False)
    _, _, _, out = run(qs, free, dtype, ids, values, rest=rest)
    check(free, ids, values, None, None, rest, out)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["ties", "equal", "falling", "rising", "stripe", "wide",
                                  "negative", "zeros"])
@pytest.mark.parametrize("V", [700, 9001, 70000])
def test_values(qs, V, kind, dtype, rest):
    """Ties, ordered rows, one lane's places on top, wide ranges, all negative."""
    print(f"distill values V={V} {kind} {dtype} rest={rest}", flush=True)
    B = 3
    z = make(V, B, V, kind)
    ids, values = teacher(np.random.default_rng(V), z, None, None, 33, rest)
    _, _, _, out = run(qs, z, dtype, ids, values, rest=rest)
    check(z, ids, values, None, None, rest, out)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 40, 3001, 70000])
def test_row_errors(qs, V, dtype, rest):
    """Every row error beside rows that are fine, and values that are legal."""
    print(f"distill errors V={V} {dtype} rest={rest}", flush=True)
    rng = np.random.default_rng(V)
    B, K = 26, 4
    z = make(5, B, V, "normal")
    T = np.ones(B, np.float32)
    legal = np.ones((B, V), bool)
    ids, values = teacher(rng, z, None, T, K, rest, pad=False)
    z[0, V - 1] = np.nan
    z[1, 0] = np.inf
    z[2, :] = -np.inf
    z[3, :] = -np.inf
    z[3, V // 2] = np.nan                  # NaN among -inf
    legal[4] = False
    z[5, V - 1] = np.nan
    legal[5, V - 1] = V == 1               # NaN at an illegal place
    T[6], T[7], T[8], T[9] = 0.0, -1.0, np.nan, np.inf
    ids[10, 0] = V
    ids[11, 3] = -2
    ids[12, 3] = np.iinfo(np.int32).min
    ids[13, 3] = np.iinfo(np.int32).max
    z[14, : V // 2] = -np.inf              # legal -inf tokens
    T[15] = 1e-38
    T[16] = 3e38
    ids[17] = -1
    ids[18, 0] = ids[18, 3] = 0            # a token named twice
    ids[18, 1:3] = -1
    values[18] = -1.0
    ids[19, 1] = ids[19, 2] = V - 1
    ids[19, 0] = ids[19, 3] = -1
    legal[19, V - 1] = False               # twice, and illegal
    z[20, ids[20, np.argmax(ids[20] >= 0)]] = np.nan   # a listed token's logit
    z[21, ids[21, np.argmax(ids[21] >= 0)]] = np.inf
    values[22, np.argmax(ids[22] >= 0)] = np.nan
    values[23, np.argmax(ids[23] >= 0)] = np.inf
    values[24, np.argmax(ids[24] >= 0)] = 1.5          # no log-probability
    values[25] = -np.inf                   # a teacher without any weight
    _, _, _, out = run(qs, z, dtype, ids, values, T, legal, rest)
    check(z, ids, values, T, legal, rest, out)


def test_illegal_slots_count_as_empty(qs):
    """What a slot of an illegal token holds is not read, nor what an empty one holds;
    the gradient does not reach them."""
    z = make(11, 4, 5003, "normal")
    legal = np.random.default_rng(11).random((4, 5003)) < 0.5
    legal[:, :4] = [True, False, True, False]
    ids = np.tile(np.array([0, 1, 2, 3, -1], np.int32), (4, 1))
    for bad in (np.nan, np.inf, -np.inf, 50.0):
        for rest in (False, True):
            values = np.array([[-1.0, bad, -2.0, bad, bad]] * 4, np.float32)
            none = np.where(np.isin(ids, (1, 3)), -1, ids).astype(np.int32)
            _, a = check_grad(qs, z, "f32", ids, values, None, legal, rest, np.ones(4, np.float32))
            _, _, _, out = run(qs, z, "f32", ids, values, None, legal, rest)
            check(z, ids, values, None, legal, rest, out)
            _, _, _, same = run(qs, z, "f32", none, values, None, legal, rest)
            assert all((out[k] == same[k]).all() for k in out)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("K", [1, 2, 63, 64, 65, 255, 257, 700, 1024])
@pytest.mark.parametrize("V", [1024, 70001])
def test_long_lists(qs, V, K, rest):
    """Lists up to the longest; with V = K every token is listed."""
    print(f"distill V={V} K={K} rest={rest}", flush=True)
    rng = np.random.default_rng(K)
    for dtype in ("f32", "bf16"):
        z = make(K, 3, V, "normal")
        ids, values = teacher(rng, z, None, None, K, rest, pad=K < V)
        _, _, _, out = run(qs, z, dtype, ids, values, rest=rest)
        check(z, ids, values, None, None, rest, out)


@pytest.mark.parametrize("B,V", [(1, 151936), (2, 600), (300, 2000), (1500, 777), (70, 40000)])
def test_batches(qs, B, V):
    """From one long row (spread over the GPU) to more rows than compute units; the same
    call twice gives the same bits."""
    import torch
    print(f"distill batch B={B} V={V}", flush=True)
    z = make(B, B, V, "normal")
    ids, values = teacher(np.random.default_rng(B), z, None, None, 9, True)
    for dtype in ("f32", "bf16"):
        _, _, _, out = run(qs, z, dtype, ids, values, rest=True)
        check(z, ids, values, None, None, True, out)
        _, _, _, again = run(qs, z, dtype, ids, values, rest=True)
        for k in out:
            assert torch.equal(out[k].view(torch.int32), again[k].view(torch.int32)), k


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 3001, 100003])
def test_temperatures(qs, V, dtype, rest):
    """Every power of ten that a temperature can be, beside waves and parts without a
    legal or a finite token."""
    print(f"distill temperatures V={V} {dtype} rest={rest}", flush=True)
    T = np.repeat(10.0 ** np.arange(-37, 39), 3).astype(np.float32)
    B = T.size
    z, legal = gap_rows(V, B, V)
    rng = np.random.default_rng(V)
    ids, values = teacher(rng, z[:, :], legal, T, 6, rest)
    _, _, _, out = run(qs, z, dtype, ids, values, T, legal, rest)
    check(z, ids, values, T, legal, rest, out)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 3001, 100003])
def test_large_logits(qs, V, dtype, rest):
    """Logits up to 1e37 as they are and at temperatures of their own size."""
    print(f"distill large logits V={V} {dtype}", flush=True)
    e = np.repeat(np.arange(0, 37), 2)
    B = e.size
    z, legal = gap_rows(V, B, V)
    ids, values = teacher(np.random.default_rng(V), z, legal, None, 6, rest)
    z = bf16(z * (10.0 ** e)[:, None])
    T = np.where(np.arange(B) % 2 == 0, 1.0, 10.0 ** e).astype(np.float32)
    _, _, _, out = run(qs, z, dtype, ids, values, T, legal, rest)
    check(z, ids, values, T, legal, rest, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 3001, 70001])
def test_lowest_values(qs, V, dtype):
    """The type's lowest value as a mask: such tokens are finite, weigh nothing beside
    others, and share a row that holds nothing else."""
    low = np.float32(-3.3895314e38)  # bf16's lowest
    z = make(V, 4, V, "normal")
    z[0, V // 2:] = low
    z[1] = low
    z[2] = low
    z[2, 1] = 0.0
    z[3, 0] = low
    ids = np.array([[0, 1, V - 1], [0, 1, V - 1], [0, 2, V - 1], [0, 1, 2]], np.int32)
    values = np.log(np.array([[0.5, 0.25, 0.125]] * 4)).astype(np.float32)
    for rest in (False, True):
        lg, t, d, out = run(qs, z, dtype, ids, values, rest=rest)
        check(z, ids, values, None, None, rest, out)
        check_grad(qs, z, dtype, ids, values, None, None, rest, np.ones(4, np.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [45, 3001, 70001])
def test_bits_past_the_row_are_ignored(qs, V, dtype):
    import torch
    z = make(V, 3, V, "normal")
    legal = np.random.default_rng(V).random((3, V)) < 0.5
    legal[:, :3] = True
    ids, values = teacher(np.random.default_rng(1), z, legal, None, 8, True)
    words = pack(legal)
    full = words.copy().view(np.uint32)
    if V % 32:
        full[:, -1] |= np.uint32((0xFFFFFFFF << (V % 32)) & 0xFFFFFFFF)
    lg = on_gpu(z, dtype, extra=3)
    t, _ = args_of(ids, values)
    outs = [qs.distill_loss(lg, *t, rest=True, bitmask=torch.from_numpy(w.view(np.int32)).cuda())
            for w in (words, full)]
    for k in outs[0]:
        assert torch.equal(outs[0][k], outs[1][k]), k
    check(z, ids, values, None, legal, True, outs[1])


# --------------------------------------------------------------------------

def check_grad(qs, z, dtype, ids, values, T, legal, rest, g, extra=0, **kw):
    """The gradient against the formula, from the forward call's state."""
    import torch
    lg, t, d, out = run(qs, z, dtype, ids, values, T, legal, rest, extra)
    grad = qs.distill_loss_backward(lg, *t, out["state"], out["status"],
                                    torch.from_numpy(g).cuda(), rest=rest, **d, **kw)
    torch.cuda.synchronize()
    compare_grad(z, dtype, ids, values, T, legal, rest, g, out, grad)
    return out, grad


def compare_grad(z, dtype, ids, values, T, legal, rest, g, out, grad):
    B, V = z.shape
    half = U if dtype == "f32" else 2.0 ** -8
    got = grad.float().cpu().numpy().astype(np.float64)
    status = out["status"].cpu().numpy()
    states = out["state"].cpu().numpy().astype(np.float64)
    for r in range(B):
        if status[r] != oracle.ROW_OK:
            assert (got[r] == 0).all(), r
            continue
        Tr = 1.0 if T is None else float(T[r])
        ok = np.ones(V, bool) if legal is None else legal[r]
        want = oracle.distill_grad_row(z[r], ok, Tr, ids[r], values[r], rest, g[r], states[r])
        assert (got[r][~ok] == 0).all(), r
        with np.errstate(over="ignore", invalid="ignore"):
            a = np.where(ok, (z[r].astype(np.float64) - states[r][2]) / Tr, 0.0)
        a = np.clip(a, -1e4, 0.0)
        by = abs(float(g[r])) / Tr
        c = by * abs(states[r][4])
        tok = ids[r][ids[r] >= 0]
        tol = U * (8 * np.abs(a) + 8 * abs(states[r][3]) + 16) * np.abs(want)
        tol[tok] = D * by * (2 + abs(states[r][7]))
        # a weight below the least normal float32 may be taken as 0, and so may an element
        tol = tol + 2.0 ** -126 * (1 + c) + (half + U) * np.abs(want)
        big = np.abs(want) > 3e38
        assert (np.abs(got[r][big]) > 2.9e38).all() and (got[r][big] * want[big] > 0).all(), r
        bad = ~big & ~(np.abs(got[r] - want) <= 1.01 * tol)
        assert not bad.any(), (r, np.nonzero(bad)[0][:4], got[r][bad][:4], want[bad][:4],
                               tol[bad][:4])


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", SIZES)
def test_grad_sizes(qs, V, dtype, rest):
    print(f"distill grad V={V} {dtype} rest={rest}", flush=True)
    rng = np.random.default_rng(V)
    B = 6
    z = make(V, B, V, "normal")
    legal = rng.random((B, V)) < 0.4
    legal[0] = True
    legal[3] = False
    z[~legal] = np.array([np.nan, np.inf, 3e38, -np.inf], np.float32)[
        rng.integers(0, 4, (~legal).sum())]
    T = rng.uniform(0.3, 2.0, B).astype(np.float32)
    g = rng.normal(0, 1, B).astype(np.float32)
    for K in (1, 70):
        ids, values = teacher(rng, z, legal, T, K, rest)
        ids[5], values[5] = -1, np.nan
        _, grad = check_grad(qs, z, dtype, ids, values, T, legal, rest, g, extra=1)
        if not rest:
            assert bool((grad[5] == 0).all())
    free = make(V + 1, B, V, "normal")
    ids, values = teacher(rng, free, None, None, 20, rest, pad=False)
    check_grad(qs, free, dtype, ids, values, None, None, rest, g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 64, 257, 1024])
def test_grad_long_lists(qs, K, dtype):
    """Lists spread over the row, beside each other, and of every token."""
    print(f"distill grad K={K} {dtype}", flush=True)
    rng = np.random.default_rng(K)
    for V in (1024, 40003):
        z = make(K, 4, V, "normal")
        ids, values = teacher(rng, z, None, None, K, True, pad=False)
        ids[1] = V - K + np.arange(K)
        ids[2] = np.arange(K)[::-1]
        g = rng.normal(0, 1, 4).astype(np.float32)
        for rest in (False, True):
            check_grad(qs, z, dtype, ids, values, None, None, rest, g)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 3001, 40003])
def test_grad_temperatures_and_large_logits(qs, V, dtype, rest):
    """Every power of ten that a temperature can be; logits up to 1e37 as they are and at
    temperatures of their own size; incoming gradients up to the largest."""
    print(f"distill grad temperatures V={V} {dtype} rest={rest}", flush=True)
    T = np.repeat(10.0 ** np.arange(-37, 39), 3).astype(np.float32)
    B = T.size
    rng = np.random.default_rng(V)
    z, legal = gap_rows(V, B, V)
    ids, values = teacher(rng, z, legal, T, 6, rest)
    g = rng.normal(0, 1, B).astype(np.float32)
    check_grad(qs, z, dtype, ids, values, T, legal, rest, g)
    e = np.repeat(np.arange(0, 37), 2)
    B = e.size
    z, legal = gap_rows(V, B, V)
    ids, values = teacher(rng, z, legal, None, 6, rest)
    z = bf16(z * (10.0 ** e)[:, None])
    T = np.where(np.arange(B) % 2 == 0, 1.0, 10.0 ** e).astype(np.float32)
    g = np.where(np.arange(B) % 4 < 2, 1.0, 3e38).astype(np.float32)
    check_grad(qs, z, dtype, ids, values, T, legal, rest, g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grad_in_place_and_padding(qs, dtype):
    """The gradient over its own logits, and what lies behind a row's last token."""
    import torch
    V = 8195
    rng = np.random.default_rng(2)
    z = make(2, 5, V, "normal")
    ids, values = teacher(rng, z, None, None, 30, True)
    g = rng.normal(0, 1, 5).astype(np.float32)
    out, want = check_grad(qs, z, dtype, ids, values, None, None, True, g)
    lg = on_gpu(z, dtype, extra=2)
    base = lg._base if lg._base is not None else lg
    behind = base[:, V:].clone()
    t, _ = args_of(ids, values)
    got = qs.distill_loss_backward(lg, *t, out["state"], out["status"],
                                   torch.from_numpy(g).cuda(), rest=True, out=lg)
    torch.cuda.synchronize()
    assert got.data_ptr() == lg.data_ptr()
    assert torch.equal(got, want)
    assert torch.equal(base[:, V:], behind)


@pytest.mark.parametrize("rest", [False, True])
def test_gradient_against_differences(qs, rest):
    """Central differences of the loss in fp64 (the oracle's), which the formula's
    gradient meets to the differences' own error."""
    rng = np.random.default_rng(7)
    V, K, h = 50, 6, 1e-5
    z = make(7, 4, V, "normal")
    legal = rng.random((4, V)) < 0.7
    legal[:, :2] = True
    T = np.array([1.0, 0.5, 1.7, 1.0], np.float32)
    ids, values = teacher(rng, z, legal, T, K, rest)
    g = np.ones(4, np.float32)
    _, grad = check_grad(qs, z, "f32", ids, values, T, legal, rest, g)
    got = grad.cpu().numpy()
    for r in range(4):
        for i in range(V):
            lo, hi = z[r].astype(np.float64).copy(), z[r].astype(np.float64).copy()
            lo[i] -= h
            hi[i] += h
            f = [oracle.distill_row(x, legal[r], T[r], ids[r], values[r], rest)["loss"]
                 for x in (lo, hi)]
            d = (f[1] - f[0]) / (2 * h)
            # third derivatives are below 1 / T^3, rounding 2^-52 |loss| / h
            tol = h * h / T[r] ** 3 + 2.0 ** -50 * (abs(f[0]) + 10) / h + 2.0 ** -20 * abs(d) + 1e-6
            assert abs(got[r, i] - d) <= tol, (r, i, got[r, i], d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 1000, 32003, 100001])
def test_peaked_rows(qs, V, dtype):
    """Teacher and student almost certain of one token (listed, or of the rest): the
    loss and the gradient keep the relative precision of what is left."""
    print(f"distill peaked V={V} {dtype}", flush=True)
    rng = np.random.default_rng(V)
    up = np.array([12.0, 16.0, 20.0, 26.0, 34.0, 60.0])
    B = up.size
    z = rng.normal(0, 2, (B, V))
    at = rng.integers(0, V, B)
    z[np.arange(B), at] = up
    z = bf16(z)
    other = (at[:, None] + 1 + np.arange(3)) % V
    for listed in (True, False):
        ids = np.concatenate((at[:, None] if listed else (at[:, None] + 4) % V, other), 1)
        ids = ids.astype(np.int32)
        for rest in (False, True):
            if rest and listed:
                small = np.exp(-up)[:, None] * np.array([0.5, 1.0, 2.0])
                first = np.log1p(-4 * np.exp(-up))[:, None]
                values = np.concatenate((first, np.log(small)), 1).astype(np.float32)
            elif rest:
                values = np.log(np.exp(-up)[:, None] * np.array([0.5, 1, 2, 1])).astype(np.float32)
            else:
                values = np.take_along_axis(z, ids.astype(np.int64), 1) * np.float32(1.125)
            _, _, _, out = run(qs, z, dtype, ids, values, rest=rest)
            check(z, ids, values, None, None, rest, out)
            check_grad(qs, z, dtype, ids, values, None, None, rest, np.ones(B, np.float32))


def test_teacher_above_one(qs):
    """Stored log-probabilities whose rounding adds up to more than 1 leave nothing to
    the rest; the loss and its gradient follow the values as they are."""
    z = make(3, 3, 500, "normal")
    ids = np.tile(np.arange(4, dtype=np.int32), (3, 1))
    values = np.log(np.array([[0.5, 0.3, 0.2, 0.05], [1.0, 0.004, 0, 0], [2.5, 0.0, 0.0, 0.1]]),
                    where=np.array([[True] * 4, [True, True, False, False],
                                    [True, False, False, True]]),
                    out=np.full((3, 4), -np.inf)).astype(np.float32)
    _, _, _, out = run(qs, z, "f32", ids, values, rest=True)
    check(z, ids, values, None, None, True, out)
    check_grad(qs, z, "f32", ids, values, None, None, True, np.ones(3, np.float32))


def test_own_top_lists_as_teacher(qs):
    """token_logprobs' top tokens are a teacher's lists as they are: a row against itself
    has no loss and no gradient, and rows with fewer tokens than slots are padded."""
    import torch
    V, n = 30011, 20
    z = make(9, 6, V, "normal")
    legal = np.random.default_rng(9).random((6, V)) < 0.5
    legal[0], legal[0, 5:9] = False, True
    lg = on_gpu(z, "f32")
    T = torch.full((6,), 0.8, device="cuda")
    bm = torch.from_numpy(pack(legal)).cuda()
    tok = torch.zeros(6, dtype=torch.int32, device="cuda")
    top = qs.token_logprobs(lg, tok, temperature=T, bitmask=bm, top_n=n)
    out = qs.distill_loss(lg, top["top_ids"], top["top_logprobs"], temperature=T, bitmask=bm,
                          rest=True)
    grad = qs.distill_loss_backward(lg, top["top_ids"], top["top_logprobs"], out["state"],
                                    out["status"], torch.ones(6, device="cuda"), temperature=T,
                                    bitmask=bm, rest=True)
    # log-probabilities of about 10 are off by some 2^-20 each; the loss is of second
    # order in them, but for sum q - 1, which the rest takes
    assert bool((out["loss"].abs() < 1e-5).all())
    assert bool((grad.abs() < 1e-5).all())
    check(z, top["top_ids"].cpu().numpy(), top["top_logprobs"].cpu().numpy(),
          T.cpu().numpy(), legal, True, out)


# --------------------------------------------------------------------------

def test_autograd(qs):
    """loss carries a gradient to the logits, the other outputs do not."""
    import torch
    rng = np.random.default_rng(4)
    z = make(4, 5, 3001, "normal")
    ids, values = teacher(rng, z, None, None, 12, True)
    t, _ = args_of(ids, values)
    T = torch.rand(5, device="cuda") + 0.5
    for dtype in ("f32", "bf16"):
        leaf = on_gpu(z, dtype).detach().requires_grad_()
        out = qs.distill_loss(leaf, *t, temperature=T, rest=True)
        assert out["loss"].requires_grad
        assert not out["state"].requires_grad and not out["status"].requires_grad
        w = torch.randn(5, device="cuda")
        (grad,) = torch.autograd.grad((out["loss"] * w).sum(), leaf, retain_graph=True)
        want = qs.distill_loss_backward(leaf.detach(), *t, out["state"], out["status"], w,
                                        temperature=T, rest=True)
        assert grad.dtype is leaf.dtype and torch.equal(grad, want)
        # an expanded incoming gradient, a call without one, a second derivative
        (mean,) = torch.autograd.grad(out["loss"].mean(), leaf, retain_graph=True)
        assert bool(torch.isfinite(mean).all())
        (g,) = torch.autograd.grad(out["loss"].sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(g.float().sum(), leaf)
        with torch.no_grad():
            assert not qs.distill_loss(leaf, *t, rest=True)["loss"].requires_grad
        # logits changed in place after the call: the backward pass says so
        held = torch.randn(5, 3008, device="cuda").to(leaf.dtype).requires_grad_()
        moved = (held * 1.0)[:, :3001]
        loss = qs.distill_loss(moved, *t, rest=True)["loss"]
        with torch.no_grad():
            moved.add_(1.0)
        with pytest.raises(RuntimeError):
            loss.sum().backward()


def test_autograd_outputs_in_place(qs):
    """The losses may be changed in place (a masked or weighted sum does so); the state,
    which the gradient reads, may not: torch reports it."""
    import torch
    z = torch.randn(4, 512, device="cuda")
    ids = torch.tensor([[1, 500, -1, 3]] * 4, dtype=torch.int32, device="cuda")
    val = torch.rand(4, 4, device="cuda").log()
    w = torch.tensor([1.0, 0.0, 2.0, -1.0], device="cuda")
    grads = []
    for in_place in (False, True):
        lg = z.clone().requires_grad_()
        loss = qs.distill_loss(lg, ids, val)["loss"]
        if in_place:
            loss *= w
        else:
            loss = loss * w
        loss.sum().backward()
        grads.append(lg.grad)
    assert torch.equal(*grads) and bool(grads[0].any())
    with pytest.raises(RuntimeError):
        out = qs.distill_loss(z.clone().requires_grad_(), ids, val)
        out["state"].mul_(2.0)
        out["loss"].sum().backward()


def test_refusals(qs):
    import torch
    B, V, K = 3, 100, 4
    lg = torch.randn(B, 104, device="cuda")[:, :V]
    ids = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    ids[:] = torch.arange(K, device="cuda")
    val = torch.zeros(B, K, device="cuda")
    ok = qs.distill_loss(lg, ids, val)
    bad = [dict(logits=lg.cpu()), dict(logits=lg[0]), dict(logits=torch.randn(V, B, device="cuda").t()),
           dict(ids=ids.long()), dict(ids=ids[:2]), dict(ids=ids[0]), dict(ids=ids.cpu()),
           dict(ids=torch.zeros(B, 2 * K, dtype=torch.int32, device="cuda")[:, ::2]),
           dict(val=val.double()), dict(val=val[:, :2]), dict(val=val.cpu()),
           dict(val=val.clone().requires_grad_()),
           dict(temperature=torch.ones(B)), dict(temperature=torch.ones(B - 1, device="cuda")),
           dict(bitmask=torch.zeros(B, 4, dtype=torch.int64, device="cuda")),
           dict(workspace=torch.empty(8, dtype=torch.uint8))]
    for kw in bad:
        kw = dict(kw)
        args = (kw.pop("logits", lg), kw.pop("ids", ids), kw.pop("val", val))
        with pytest.raises(ValueError):
            qs.distill_loss(*args, **kw)
    with pytest.raises((TypeError, RuntimeError)):
        qs.distill_loss(lg.half(), ids, val)
    with pytest.raises(RuntimeError):
        qs.distill_loss(lg, torch.zeros(B, 1025, dtype=torch.int32, device="cuda"),
                        torch.zeros(B, 1025, device="cuda"))
    with pytest.raises(RuntimeError):
        qs.distill_loss(lg, ids[:, :0].contiguous(), val[:, :0].contiguous())
    with pytest.raises(RuntimeError):
        qs.distill_loss(torch.randn(B, 101, device="cuda")[:, :V], ids, val)
    with pytest.raises(RuntimeError):
        qs.distill_loss(lg, ids, val, bitmask=torch.zeros(B, 3, dtype=torch.int32, device="cuda"))
    g = torch.ones(B, device="cuda")
    back = (lg, ids, val, ok["state"], ok["status"], g)
    qs.distill_loss_backward(*back)
    for at, t in ((3, ok["state"][:, :7]), (3, ok["state"].double()), (4, ok["status"].float()),
                  (5, g[:2]), (5, g.double()), (5, g.cpu())):
        args = list(back)
        args[at] = t
        with pytest.raises(ValueError):
            qs.distill_loss_backward(*args)
    for out in (torch.empty(B, V, dtype=torch.bfloat16, device="cuda"),
                torch.empty(B, V + 1, device="cuda"), torch.empty(B, V),
                torch.empty(V, B, device="cuda").t(),
                torch.empty(B, V, device="cuda").requires_grad_()):
        with pytest.raises(ValueError):
            qs.distill_loss_backward(*back, out=out)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(lg, torch.ones_like(lg))
        with pytest.raises(ValueError):
            qs.distill_loss(dual, ids, val)
        with pytest.raises(ValueError):
            qs.distill_loss_backward(dual, *back[1:])


def test_temperature_gets_no_gradient(qs):
    """A temperature that asks for a gradient is refused, not left without one; outside
    of grad mode it is a number like any other."""
    import torch
    lg = torch.randn(2, 64, device="cuda")
    ids = torch.arange(4, dtype=torch.int32, device="cuda").repeat(2, 1)
    val = torch.zeros(2, 4, device="cuda")
    T = torch.full((2,), 0.7, device="cuda", requires_grad=True)
    for z in (lg, lg.clone().requires_grad_()):
        with pytest.raises(ValueError, match="temperature"):
            qs.distill_loss(z, ids, val, temperature=T)
    want = qs.distill_loss(lg, ids, val, temperature=T.detach())
    with torch.no_grad():
        got = qs.distill_loss(lg, ids, val, temperature=T)
        qs.distill_loss_backward(lg, ids, val, got["state"], got["status"],
                                 torch.ones(2, device="cuda"), temperature=T)
    assert torch.equal(got["loss"], want["loss"])


def test_empty_batch(qs):
    import torch
    for V in (64, 70016):
        lg = torch.empty(0, V, device="cuda")
        ids = torch.empty(0, 4, dtype=torch.int32, device="cuda")
        val = torch.empty(0, 4, device="cuda")
        assert qs.distill_loss_workspace_for(lg) is None
        out = qs.distill_loss(lg, ids, val)
        assert out["loss"].shape == (0,) and out["state"].shape == (0, 8)
        grad = qs.distill_loss_backward(lg, ids, val, out["state"], out["status"],
                                        torch.empty(0, device="cuda"))
        assert grad.shape == (0, V)
        leaf = lg.clone().requires_grad_()
        qs.distill_loss(leaf, ids, val)["loss"].sum().backward()
        assert leaf.grad.shape == (0, V)


def test_most_rows(qs):
    """The largest batch, 2^22 - 1 rows of 7 tokens, two of them listed. Five terms of S_R,
    so e_S is at most 32 units; a loss is at most 60 or so, a gradient element at most 1."""
    import torch
    B, V = (1 << 22) - 1, 7
    torch.manual_seed(3)
    z = torch.randn(B, 8, device="cuda").mul_(3).bfloat16()[:, :V]
    ids = torch.tensor([[4, 1]], dtype=torch.int32, device="cuda").expand(B, 2).contiguous()
    q = torch.rand(B, 2, device="cuda") * 0.45 + 0.01
    out = qs.distill_loss(z, ids, q.log(), rest=True)
    assert not out["status"].any()
    lp = torch.log_softmax(z.double(), 1)
    at = ids.long()
    # the probabilities that the float32 logarithms stand for
    q = q.log().double().exp()
    others = torch.tensor([0, 2, 3, 5, 6], device="cuda")
    lr, qr = torch.logsumexp(lp[:, others], 1), 1 - q.sum(1)
    want = (q * (q.log() - lp.gather(1, at))).sum(1) + qr * (qr.log() - lr)
    assert bool(((out["loss"] - want).abs() <= U * (32 + 2 * want.abs())).all())
    grad = qs.distill_loss_backward(z, ids, q.log().float(), out["state"], out["status"],
                                    torch.ones(B, device="cuda"), rest=True)
    want = (lp - lr[:, None]).exp() * (lr.exp() - qr)[:, None]
    want.scatter_(1, at, lp.gather(1, at).exp() - q)
    # log p of up to 30 from a state rounded to float32
    assert bool(((grad - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 128 * U).all())


def test_writes_and_inference_mode(qs):
    """The gradient written over a buffer counts as a change of it; tensors of inference
    mode are taken."""
    import torch
    B, V = 4, 512
    ids = torch.tensor([[1, 5, -1]] * B, dtype=torch.int32, device="cuda")
    val = torch.rand(B, 3, device="cuda").log()
    g = torch.ones(B, device="cuda")
    z = torch.randn(B, V, device="cuda").requires_grad_()
    kept = z.detach()
    o = qs.distill_loss(kept, ids, val)
    loss = qs.distill_loss(z, ids, val)["loss"]
    qs.distill_loss_backward(kept, ids, val, o["state"], o["status"], g, out=kept)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()
    with torch.inference_mode():
        x = torch.randn(B, V, device="cuda")
        o = qs.distill_loss(x, ids, val, rest=True)
        qs.distill_loss_backward(x, ids, val, o["state"], o["status"], g, rest=True, out=x)
    torch.cuda.synchronize()
    assert not o["status"].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grad_of_non_finite_gradients(qs, dtype):
    """A NaN or an infinity as a row's incoming gradient reaches every legal token of
    it and no other row; illegal tokens and rows with an error stay 0. Finite gradients
    past the largest value give no NaN."""
    import torch
    rng = np.random.default_rng(21)
    V, B = 5003, 8
    z = make(21, B, V, "normal")
    z[6] = -1e4
    z[6, 7] = 0.0
    legal = rng.random((B, V)) < 0.5
    legal[:, :2], legal[4] = True, False
    legal[6] = True
    ids, values = teacher(rng, z, legal, None, 8, True, pad=False)
    g = np.array([np.nan, np.inf, -np.inf, 1.0, np.nan, 0.0, 1e35, -1.0], np.float32)
    T = np.array([1, 1, 1, 1, 1, 1, 1e-9, 1], np.float32)
    for rest in (False, True):
        lg, t, d, out = run(qs, z, dtype, ids, values, T, legal, rest)
        grad = qs.distill_loss_backward(lg, *t, out["state"], out["status"],
                                        torch.from_numpy(g).cuda(), rest=rest, **d)
        got = grad.float().cpu().numpy()
        for r in range(3):
            assert not np.isfinite(got[r][legal[r]]).any(), r
            assert (got[r][~legal[r]] == 0).all(), r
        assert (got[4] == 0).all() and (got[5] == 0).all()
        assert not np.isnan(got[6]).any()
        keep = [3, 5, 7]
        compare_grad(z[keep], dtype, ids[keep], values[keep], T[keep], legal[keep], rest, g[keep],
                     {k: v[keep] for k, v in out.items()}, grad[keep])


def test_other_streams_and_workspace(qs):
    """Two calls at once on two streams; a caller's scratch memory used again; what
    cannot hold the call is refused."""
    import torch
    V, B = 151936, 40
    z = make(1, B, V, "normal")
    ids, values = teacher(np.random.default_rng(1), z, None, None, 30, True)
    lg = on_gpu(z, "bf16")
    t, _ = args_of(ids, values)
    want = qs.distill_loss(lg, *t, rest=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            o = qs.distill_loss(lg, *t, rest=True)
            outs.append((o, qs.distill_loss_backward(lg, *t, o["state"], o["status"],
                                                     torch.ones(B, device="cuda"), rest=True)))
    torch.cuda.synchronize()
    for o, _ in outs:
        assert all(torch.equal(o[k], want[k]) for k in want)
    assert torch.equal(outs[0][1], outs[1][1])
    ws = qs.distill_loss_workspace_for(lg)
    if ws is not None:
        for fill in (0, 255):
            ws.fill_(fill)
            got = qs.distill_loss(lg, *t, rest=True, workspace=ws)
            small = qs.distill_loss(lg[:3], t[0][:3], t[1][:3], rest=True, workspace=ws)
            torch.cuda.synchronize()
            assert all(torch.equal(got[k], want[k]) for k in want)
            # fewer rows may be cut into other parts: sums in another order
            assert torch.allclose(small["loss"], want["loss"][:3], rtol=1e-5, atol=1e-5)
        for bad in (ws[:-1], ws[256:]):
            with pytest.raises(RuntimeError):
                qs.distill_loss(lg, *t, rest=True, workspace=bad)


def test_graph_replays(qs):
    """Loss and gradient in one graph, replayed between eager calls on other data."""
    import torch
    V, B = 70001, 9
    rng = np.random.default_rng(6)
    sets = []
    for k in range(3):
        z = make(60 + k, B, V, "normal")
        ids, values = teacher(rng, z, None, None, 16, True)
        sets.append((on_gpu(z, "bf16"), *args_of(ids, values)[0]))
    lg, ids, val = (x.clone() for x in sets[0])
    lg = on_gpu(np.zeros((B, V), np.float32), "bf16")
    g = torch.rand(B, device="cuda")

    def step(lg, ids, val):
        o = qs.distill_loss(lg, ids, val, rest=True)
        return o["loss"], o["state"], qs.distill_loss_backward(lg, ids, val, o["state"],
                                                               o["status"], g, rest=True)

    lg.copy_(sets[0][0])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(lg, ids, val)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(lg, ids, val)
    for k in (1, 0, 2, 1):
        for a, b in zip((lg, ids, val), sets[k]):
            a.copy_(b)
        graph.replay()
        want = step(*sets[k])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), k


def test_offsets_past_32_bits(qs):
    """Rows that start past 2^32 bytes."""
    import torch
    V, B = 1 << 20, 2100
    lg = torch.zeros(B, V, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(3)
    rows = [0, 1023, 1024, 2047, 2048, 2099]
    z = make(3, len(rows), V, "normal")
    at = torch.tensor(rows, device="cuda")
    lg[at] = torch.from_numpy(z).cuda().to(torch.bfloat16)
    few, v = teacher(rng, z, None, None, 5, True)
    ids = torch.full((B, 5), -1, dtype=torch.int32, device="cuda")
    val = torch.zeros(B, 5, device="cuda")
    ids[at], val[at] = torch.from_numpy(few).cuda(), torch.from_numpy(v).cuda()
    out = qs.distill_loss(lg, ids, val, rest=True)
    g = torch.ones(B, device="cuda")
    grad = qs.distill_loss_backward(lg, ids, val, out["state"], out["status"], g, rest=True)
    torch.cuda.synchronize()
    pick = {k: x[at] for k, x in out.items()}
    check(z, few, v, None, None, True, pick)
    compare_grad(z, "bf16", few, v, None, None, True, np.ones(len(rows), np.float32), pick,
                 grad[at])


def test_longest_row(qs):
    """A row of 2^30 bf16 tokens, its last one listed."""
    import torch
    V = 1 << 30
    lg = torch.zeros(1, V, dtype=torch.bfloat16, device="cuda")
    lg[0, V - 1] = 30.0
    lg[0, 5] = 20.0
    ids = torch.tensor([[V - 1, 7]], dtype=torch.int32, device="cuda")
    val = torch.log(torch.tensor([[0.5, 0.25]], device="cuda"))
    out = qs.distill_loss(lg, ids, val, rest=True)
    S = np.exp(-30.0) * (V - 2) + np.exp(-10.0) + 1.0
    pr = (np.exp(-30.0) * (V - 3) + np.exp(-10.0)) / S
    want = 0.5 * (np.log(0.5) + np.log(S)) + 0.25 * (np.log(0.25) + 30 + np.log(S)) \
        + 0.25 * (np.log(0.25) - np.log(pr))
    # 2^30 equal terms, each lane's and then all lanes' and parts' sums
    e_S = U * (depth(V) + 64 + 8)
    assert abs(float(out["loss"][0]) - want) <= abs(pr - 0.25) * e_S + 4 * U * abs(want)
    grad = qs.distill_loss_backward(lg, ids, val, out["state"], out["status"],
                                    torch.ones(1, device="cuda"), rest=True, out=lg)
    got = grad[0, [5, 6, 7, V - 2, V - 1]].float().cpu().numpy()
    w = np.array([np.exp(-10.0), np.exp(-30.0)]) / S / pr * (pr - 0.25)
    named = np.array([np.exp(-30.0) / S - 0.25, 1.0 / S - 0.5])
    wanted = np.array([w[0], w[1], named[0], w[1], named[1]])
    assert (np.abs(got - wanted) <= (2.0 ** -8 + 2e-4) * np.abs(wanted)).all(), (got, wanted)


def few_in_a_list(rng, B, V, K, rest, span):
    """Lists of K tokens anywhere; rest: of probability 0.6 together, else logits of
    either sign up to `span`."""
    ids = np.stack([rng.permutation(V)[:K] for _ in range(B)]).astype(np.int32)
    values = np.log(0.6 * rng.dirichlet(np.ones(K), B)) if rest else rng.uniform(-span, span, (B, K))
    return ids, values.astype(np.float32)


def far_apart(V):
    """Finite logits further apart than float32's largest value, and temperatures that weigh
    them all: in any order (every wave has both ends), falling, and in two halves (waves
    and parts lie apart)."""
    T = np.repeat(np.array([1e36, 4e36, 1e37, 1e38, 1.2e38, 1.3e38, 2e38, 3.4e38], np.float32), 3)
    rng = np.random.default_rng(V)
    z = rng.uniform(-3.3e38, 3.3e38, (T.size, V))
    z[1::3] = np.linspace(3.3e38, -3.3e38, V)
    z[2::3] = np.where(np.arange(V) < V // 2, -3.3e38, 3.3e38)
    return rng, bf16(z), T


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 500, 1000, 3001, 20001, 70003])
def test_largest_temperatures(qs, V, dtype, rest):
    """Temperatures up to float32's largest value. log2(e) / T is below the least normal
    float32 from 1.2e38 on, where it is still good to 2^-22.5 of itself: 2 u |a| more than
    above, and |a| is below 5.6 there, 12 units against the 128 and more that a sum's
    tolerance has for its additions."""
    print(f"distill largest temperatures V={V} {dtype} rest={rest}", flush=True)
    rng, z, T = far_apart(V)
    ids, values = few_in_a_list(rng, T.size, V, 5, rest, 3e38)
    _, _, _, out = run(qs, z, dtype, ids, values, T, None, rest)
    check(z, ids, values, T, None, rest, out)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 1000, 3001, 40003])
def test_grad_at_largest_temperatures(qs, V, dtype, rest):
    """The same rows' gradient, incoming gradients large enough that their quotients by T are
    normal numbers; the 2 u |a| of such temperatures are within the tolerance's 8."""
    print(f"distill grad largest temperatures V={V} {dtype} rest={rest}", flush=True)
    rng, z, T = far_apart(V)
    ids, values = few_in_a_list(rng, T.size, V, 5, rest, 3e38)
    g = (1e36 * rng.normal(0, 1, T.size)).astype(np.float32)
    check_grad(qs, z, dtype, ids, values, T, None, rest, g)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 3001, 40003])
def test_grad_past_the_largest_factor(qs, V, dtype, rest):
    """Rows whose factor g (Q p_R - q_R) / T passes float32's largest value while their
    elements, each its share of it, do not: they are the formula's all the same."""
    print(f"distill grad factor V={V} {dtype} rest={rest}", flush=True)
    rng = np.random.default_rng(V)
    T = np.array([1.0, 1.0, 0.9, 1e-2, 1e-2, 1e-3, 2.0 ** -20, 1e-38], np.float32)
    g = np.array([3.4e38, -3.4e38, 3.4e38, 2e37, -2e36, 1e37, 3e33, 100.0], np.float32)
    B = T.size
    z = make(V, B, V, "normal")
    z[4:] = -2.5                           # tokens that share the mass at any temperature
    ids, values = few_in_a_list(rng, B, V, 5, rest, 3.0)
    check_grad(qs, z, dtype, ids, values, T, None, rest, g)
    legal = rng.random((B, V)) < 0.5
    legal[:, :2] = True
    check_grad(qs, z, dtype, ids, values, T, legal, rest, g)


def rows_on_gpu(seed, B, V, dtype, masked):
    """A large batch made on the GPU: its logits, mask words (or None), and a function that
    gives given rows of both as the checks take them."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind = torch.float32 if dtype == "f32" else torch.bfloat16
    lg = torch.empty(B, -(-V // 8) * 8, dtype=kind, device="cuda")
    for at in range(0, B, 64):
        lg[at:at + 64] = 3 * torch.randn(lg[at:at + 64].shape, generator=gen, device="cuda")
    words = None
    if masked:
        words = torch.randint(-2 ** 31, 2 ** 31, (B, -(-V // 32)), generator=gen, device="cuda")
        words = words.to(torch.int32)

    def rows(at):
        z = lg[at, :V].float().cpu().numpy()
        if words is None:
            return z, None
        bits = words[at].cpu().numpy().view(np.uint8)
        return z, np.unpackbits(bits, axis=1, bitorder="little")[:, :V].astype(bool)

    return lg[:, :V], words, rows


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("B,V,dtype,masked", [
    (600, 1500, "f32", False), (600, 1500, "f32", True),          # whole rows, 128 threads
    (600, 3001, "bf16", False), (600, 3001, "bf16", True),
    (600, 6000, "bf16", True), (600, 9001, "f32", False), (600, 20001, "bf16", True),
    (300, 20001, "f32", False), (300, 20001, "f32", True),        # 512 threads, 16 loads
    (300, 40003, "bf16", False), (300, 40003, "bf16", True),
    (300, 151936, "bf16", False), (300, 151936, "bf16", True),    # parts of 8 loads
    (700, 100003, "bf16", True), (200, 128259, "f32", False), (200, 128259, "f32", True),
    (600, 151936, "bf16", False),                                 # parts of 16
])
def test_many_rows(qs, B, V, dtype, masked, rest):
    """Batches that are cut in other ways than a few rows are, values of every kind of
    magnitude in every lane: some rows against the oracle, the gradient too."""
    import torch
    print(f"distill many rows B={B} V={V} {dtype} masked={masked} rest={rest}", flush=True)
    rng = np.random.default_rng(B + V)
    lg, words, rows = rows_on_gpu(B + V, B, V, dtype, masked)
    ids = ((rng.integers(0, V, B)[:, None] + np.arange(33) * (V // 40)) % V).astype(np.int32)
    ids[::3, 5:9] = -1
    values = np.log(0.7 * rng.dirichlet(np.ones(33), B)).astype(np.float32)
    T = rng.uniform(0.4, 2.0, B).astype(np.float32)
    g = rng.normal(0, 1, B).astype(np.float32)
    t, d = args_of(ids, values, T)
    d["bitmask"] = words
    out = qs.distill_loss(lg, *t, rest=rest, **d)
    grad = qs.distill_loss_backward(lg, *t, out["state"], out["status"],
                                    torch.from_numpy(g).cuda(), rest=rest, **d)
    torch.cuda.synchronize()
    assert not out["status"].any()
    at = np.unique(np.concatenate(([0, 1, B // 2, B - 2, B - 1], rng.integers(0, B, 4))))
    pick = torch.from_numpy(at).cuda()
    z, legal = rows(pick)
    some = {k: v[pick] for k, v in out.items()}
    check(z, ids[at], values[at], T[at], legal, rest, some)
    compare_grad(z, dtype, ids[at], values[at], T[at], legal, rest, g[at], some, grad[pick])


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,V", [(3, 3001), (3, 6000), (3, 9001), (3, 20001), (3, 40003),
                                 (300, 20001), (300, 40003), (600, 3001)])
def test_long_lists_of_any_row(qs, B, V, dtype, rest):
    """Lists longer than one wave's slots, worked out by all waves of a row's workgroup
    (128 to 1024 threads) or of the join's."""
    import torch
    print(f"distill long lists B={B} V={V} {dtype} rest={rest}", flush=True)
    rng = np.random.default_rng(B + V)
    lg, _, rows = rows_on_gpu(B + V, B, V, dtype, False)
    at = np.unique([0, B // 2, B - 1])
    pick = torch.from_numpy(at).cuda()
    z, _ = rows(pick)
    for K in (257, 513, 700, 1024):
        # distinct tokens, close together and far apart
        step = rng.choice([1, max(V // 1100, 1)], B)
        ids = ((rng.integers(0, V, B)[:, None] + np.arange(K) * step[:, None]) % V).astype(np.int32)
        ids = rng.permuted(ids, axis=1)
        ids[:, 100:110] = -1
        values = np.log(0.9 * rng.dirichlet(np.ones(K), B)).astype(np.float32)
        values[:, K - 1] = -np.inf
        t, _ = args_of(ids, values)
        out = qs.distill_loss(lg, *t, rest=rest)
        torch.cuda.synchronize()
        assert not out["status"].any()
        check(z, ids[at], values[at], None, None, rest, {k: v[pick] for k, v in out.items()})
        # a token named twice is found wherever its slots are
        ids[:, K - 1] = ids[:, 3]
        again = qs.distill_loss(lg, torch.from_numpy(ids).cuda(), t[1], rest=rest)
        assert bool((again["status"] == oracle.ROW_BAD_PARAM).all())


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 3001, 70003])
def test_smallest_temperatures(qs, V, dtype, rest):
    """Temperatures down to subnormal ones, 1 / T past float32's largest value: equal maxima
    share the row, the rest's or the listed tokens', and everything else has no weight."""
    print(f"distill smallest temperatures V={V} {dtype} rest={rest}", flush=True)
    T = np.repeat(np.array([2e-38, 1e-38, 3e-39, 1e-39, 1e-41, 1e-45], np.float32), 2)
    rng = np.random.default_rng(V)
    B = T.size
    z = bf16(np.minimum(make(V, B, V, "normal"), 2.0))
    ids, values = few_in_a_list(rng, B, V, 5, rest, 3.0)
    for r in range(B):
        others = np.setdiff1d(np.arange(V), ids[r])
        z[r, rng.choice(others, 3, False)] = 2.5
        if r % 2:
            z[r, ids[r, :2]] = 2.5
    _, _, _, out = run(qs, z, dtype, ids, values, T, None, rest)
    check(z, ids, values, T, None, rest, out)
    g = (T.astype(np.float64) * 1e6 * rng.uniform(1, 2, B)).astype(np.float32)
    check_grad(qs, z, dtype, ids, values, T, None, rest, g)
