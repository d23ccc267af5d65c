"""Distillation from a teacher's top tokens, its gradient, and low-rank adapters, in
fp64.

TEST INFRASTRUCTURE: only tests/, __graft_entry__.smoke() and bench.py's
cpu_baseline leg may import this module.

The definitions written out row by row: the divergence of the row's tempered, masked
softmax from the teacher's probabilities, with what neither a listed nor an illegal
token holds as one more outcome where asked; its gradient's formula; and the product
of a row's hidden state with its own adapter.
"""

import numpy as np

from .sampling import (ROW_ALL_NEG_INF, ROW_BAD_PARAM, ROW_EMPTY, ROW_NONFINITE, ROW_OK)


def _slots(z, legal, ids):
    """The slots that name a legal token: (their places in the list, their tokens)."""
    ids = np.asarray(ids, np.int64)
    live = ids >= 0
    live[live] = legal[ids[live]]
    return np.nonzero(live)[0], ids[live]


def distill_row(z, legal, T, ids, values, rest):
    """One row: z float64 [V], legal bool [V] or None, T, teacher's ids and values [K].

    Returns a dict: status, loss, state [8]; for tolerances the rest's weights w and
    exponents a (of its finite tokens), p_rest, and size, the sum of q times the
    magnitudes that loss is a difference of.
    """
    z = np.asarray(z, np.float64)
    values = np.asarray(values, np.float64)
    V = z.shape[0]
    legal = np.ones(V, bool) if legal is None else legal[:V]
    ids = np.asarray(ids, np.int64)
    out = {"loss": np.nan, "state": np.full(8, np.nan)}
    T = float(T)
    named = ids[ids >= 0]
    v = z[legal]
    if not (np.isfinite(T) and T > 0) or ((ids < -1) | (ids >= V)).any() \
            or np.unique(named).size != named.size:
        out["status"] = ROW_BAD_PARAM
        return out
    at, tok = _slots(z, legal, ids)
    t = values[at]
    if not (t <= (1.0 if rest else np.finfo(np.float32).max)).all():
        out["status"] = ROW_BAD_PARAM
    elif v.size == 0:
        out["status"] = ROW_EMPTY
    elif np.isnan(v).any() or (v == np.inf).any():
        out["status"] = ROW_NONFINITE
    elif (v == -np.inf).all():
        out["status"] = ROW_ALL_NEG_INF
    else:
        out["status"] = ROW_OK
    if out["status"] != ROW_OK:
        return out
    others = legal.copy()
    others[tok] = False
    r = z[others]
    r = r[np.isfinite(r)]
    m = v.max()
    with np.errstate(over="ignore", under="ignore"):
        d = (z[tok] - m) / T                      # the listed tokens' exponents
        e = np.exp(d)
        mr = r.max() if r.size else 0.0
        a = (r - mr) / T if r.size else np.zeros(0)
        w = np.exp(a)
        Sr = w.sum()
        dr = (mr - m) / T
        f = np.exp(dr) * Sr if r.size else 0.0
        # all weights but one maximum's own
        if (z[tok] == m).any():
            low = z[tok] < m
            more = e[low].sum() + ((~low).sum() - 1) + f
        else:
            top = np.argmax(r)
            more = e.sum() + np.delete(w, top).sum()
        ls = np.log1p(more)
        lsr = np.log1p(np.delete(w, np.argmax(r)).sum()) if r.size else 0.0
        lpr = dr + lsr - ls
        lp = d - ls
        tm = tls = qr = 0.0
        if rest:
            lq = t
            if r.size:
                qr = max(0.0, 1.0 - np.exp(lq).sum())
        else:
            if t.size and t.max() > -np.inf:
                tm = t.max()
                x = (t - tm) / T
                first = np.argmax(x)
                tls = np.log1p(np.exp(np.delete(x, first)).sum())
            lq = (t - tm) / T - tls
        q = np.exp(lq)
        Q = q.sum() + qr
        if not rest:
            Q = 1.0 if q.sum() > 0 else 0.0
        on = q > 0
        loss = (q[on] * (lq[on] - lp[on])).sum()
        size = (q[on] * (np.abs(lq[on]) + np.abs(d[on]) + abs(ls))).sum()
        if qr > 0:
            loss += qr * (np.log(qr) - lpr)
            size += qr * (abs(np.log(qr)) + abs(dr) + abs(lsr) + abs(ls))
        pr = np.exp(lpr) if r.size else 0.0
        if not r.size:
            rg = 0.0
        elif pr < 0.5:
            rg = Q * pr - qr
        else:
            rg = Q - qr - Q * np.exp(lp).sum()
    out["loss"] = loss
    out["state"] = np.array([m, ls, mr, lsr, rg, tm, tls, Q - 1.0])
    out.update(w=w, a=a, p_rest=pr, size=size, mass=Q)
    return out


def distill_grad_row(z, legal, T, ids, values, rest, g, state):
    """The gradient's formula for one row from given row statistics (float64)."""
    z = np.asarray(z, np.float64)
    V = z.shape[0]
    legal = np.ones(V, bool) if legal is None else legal[:V]
    T = float(T)
    m, ls, mr, lsr, rg, tm, tls, over = np.asarray(state, np.float64)
    out = np.zeros(V)
    at, tok = _slots(z, legal, ids)
    t = np.asarray(values, np.float64)[at]
    others = legal.copy()
    others[tok] = False
    with np.errstate(over="ignore", under="ignore"):
        out[others] = np.exp((z[others] - mr) / T - lsr) * rg
        lp = (z[tok] - m) / T - ls
        lq = t if rest else (t - tm) / T - tls
        out[tok] = over + (1.0 + over) * np.expm1(lp) - np.expm1(lq)
    return out * (float(g) / T)


def adapted_row(z, x, down, up, scale):
    """One row's logits moved by its adapter (None: none), in float64."""
    z = np.asarray(z, np.float64)
    if down is None:
        return z
    return z + float(scale) * (np.asarray(up, np.float64)
                               @ (np.asarray(down, np.float64) @ np.asarray(x, np.float64)))
