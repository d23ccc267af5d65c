"""Token log-probabilities, their gradient and the 4-bit output head in fp64.

TEST INFRASTRUCTURE: only tests/, __graft_entry__.smoke() and bench.py's
cpu_baseline leg may import this module.

The definitions written out row by row: the tempered, masked softmax of one row
in fp64, its log-probabilities, entropy and largest tokens by a stable sort,
the gradient's formula, and the head as a product with the weights the codes
stand for.
"""

import numpy as np

from .sampling import (ROW_ALL_NEG_INF, ROW_BAD_PARAM, ROW_EMPTY, ROW_NONFINITE, ROW_OK)


def score_row(z, legal, T, tokens, top_n=0):
    """One row: z float64 [V], legal bool [V] or None, T, tokens int [G].

    Returns a dict: status, logprobs [G], row_max, log_sum, entropy, top_ids,
    top_logprobs, and for tolerances a (the legal tokens' (z - m) / T) and p.
    """
    z = np.asarray(z, np.float64)
    V = z.shape[0]
    legal = np.ones(V, bool) if legal is None else legal[:V]
    tokens = np.asarray(tokens, np.int64)
    out = {"logprobs": np.where(tokens == -1, 0.0, np.nan), "row_max": np.nan, "log_sum": np.nan,
           "entropy": np.nan, "top_ids": np.full(top_n, -1, np.int64),
           "top_logprobs": np.full(top_n, -np.inf)}
    ids = np.nonzero(legal)[0]
    v = z[ids]
    if not (np.isfinite(T) and T > 0) or ((tokens < -1) | (tokens >= V)).any():
        out["status"] = ROW_BAD_PARAM
    elif ids.size == 0:
        out["status"] = ROW_EMPTY
    elif np.isnan(v).any() or (v == np.inf).any():
        out["status"] = ROW_NONFINITE
    elif (v == -np.inf).all():
        out["status"] = ROW_ALL_NEG_INF
    else:
        out["status"] = ROW_OK
    if out["status"] != ROW_OK:
        return out
    m = v.max()
    with np.errstate(over="ignore"):
        a = (v - m) / float(T)
    e = np.exp(a)
    S = e.sum()
    lse = np.log(S)
    fin = e > 0
    out["row_max"], out["log_sum"] = m, lse
    out["a"], out["p"] = a, e / S
    out["entropy"] = lse - (e[fin] * a[fin]).sum() / S
    full = np.full(V, -np.inf)
    full[ids] = a - lse
    out["full"] = full
    given = tokens >= 0
    out["logprobs"][given] = full[tokens[given]]
    order = ids[np.argsort(-v, kind="stable")]
    order = order[np.isfinite(z[order])][:top_n]
    out["top_ids"][:order.size] = order
    out["top_logprobs"][:order.size] = full[order]
    return out


def grad_row(z, legal, T, tokens, gl, gH, row_max, log_sum, entropy):
    """The gradient's formula for one row from given row statistics (float64)."""
    z = np.asarray(z, np.float64)
    V = z.shape[0]
    legal = np.ones(V, bool) if legal is None else legal[:V]
    T = float(T)
    out = np.zeros(V)
    with np.errstate(over="ignore"):
        lp = (z[legal] - float(row_max)) / T - float(log_sum)
    p = np.exp(lp)
    tokens = np.asarray(tokens, np.int64)
    live = (tokens >= 0) & (tokens < V)
    gl = np.where(live, np.asarray(gl, np.float64), 0.0)
    d = -p * gl.sum()
    if gH is not None:
        fin = p > 0
        d[fin] -= float(gH) * p[fin] * (lp[fin] + float(entropy))
    out[legal] = d
    for t, g in zip(tokens[live], gl[live]):
        if legal[t]:
            out[t] += g
    return out / T


def head_weights(codes, scales, zeros, group):
    """The weights [V, K] that the codes stand for, float64."""
    codes = np.asarray(codes)
    V, half = codes.shape
    q = np.empty((V, 2 * half))
    q[:, 0::2] = codes & 15
    q[:, 1::2] = codes >> 4
    zero = 8.0 if zeros is None else np.repeat(np.asarray(zeros, np.float64), group, 1)
    return (q - zero) * np.repeat(np.asarray(scales, np.float64), group, 1)
