"""The distillation and adapter oracle against closed forms and differences (CPU)."""

import math

import numpy as np
import pytest

import oracle


def softmax(z, T=1.0):
    e = np.exp((z - z.max()) / T)
    return e / e.sum()


def test_every_token_listed_is_the_divergence_of_two_softmaxes():
    rng = np.random.default_rng(0)
    z, t = rng.normal(0, 2, 40), rng.normal(0, 2, 40)
    for T in (0.5, 1.0, 3.0):
        p, q = softmax(z, T), softmax(t, T)
        want = (q * np.log(q / p)).sum()
        order = rng.permutation(40)
        got = oracle.distill_row(z, None, T, order, t[order], False)
        assert abs(got["loss"] - want) < 1e-12 and got["state"][7] == 0.0
        got = oracle.distill_row(z, None, T, order, np.log(q[order]), True)
        assert abs(got["loss"] - want) < 1e-9


def test_worked_example():
    """p = (1/2, 1/4, 1/8, 1/8); the teacher names the first with 1/2 and the third with
    1/4 and leaves 1/4 to the others, who have 3/8: (1/4) ln 2 + (1/4) ln (2/3)."""
    z = np.log([0.5, 0.25, 0.125, 0.125])
    got = oracle.distill_row(z, None, 1.0, [0, 2, -1], [math.log(0.5), math.log(0.25), np.nan],
                             True)
    assert abs(got["loss"] - (0.25 * math.log(2) + 0.25 * math.log(2 / 3))) < 1e-14
    assert abs(got["p_rest"] - 0.375) < 1e-14
    assert abs(got["state"][4] - 0.125) < 1e-14     # p_R - q_R
    # over the listed tokens alone: q = (2/3, 1/3) against p
    got = oracle.distill_row(z, None, 1.0, [0, 2, -1], [math.log(0.5), math.log(0.25), np.nan],
                             False)
    want = 2 / 3 * math.log(2 / 3 / 0.5) + 1 / 3 * math.log(1 / 3 / 0.125)
    assert abs(got["loss"] - want) < 1e-14
    # with the second token illegal p = (2/3, 0, 1/6, 1/6)
    legal = np.array([True, False, True, True])
    got = oracle.distill_row(z, legal, 1.0, [0, 1, 2], np.log([0.5, 0.25, 0.25]), True)
    want = 0.5 * math.log(0.75) + 0.25 * math.log(1.5) + 0.25 * math.log(1.5)
    assert abs(got["loss"] - want) < 1e-14


def test_statuses_and_rows_without_a_teacher():
    z = np.zeros(5)
    ok = oracle.ROW_OK
    none = oracle.distill_row(z, None, 1.0, [-1, -1], [np.nan, np.nan], False)
    assert none["status"] == ok and none["loss"] == 0 and none["state"][7] == -1
    alone = oracle.distill_row(z, None, 1.0, [-1], [np.nan], True)
    assert alone["status"] == ok and abs(alone["loss"]) < 1e-15
    for T, ids, values, rest, want in (
            (0.0, [0], [0.0], False, oracle.ROW_BAD_PARAM),
            (1.0, [5], [0.0], False, oracle.ROW_BAD_PARAM),
            (1.0, [-2], [0.0], False, oracle.ROW_BAD_PARAM),
            (1.0, [1, 1], [0.0, 0.0], False, oracle.ROW_BAD_PARAM),
            (1.0, [1], [np.nan], False, oracle.ROW_BAD_PARAM),
            (1.0, [1], [1.5], True, oracle.ROW_BAD_PARAM),
            (1.0, [1], [1.5], False, ok), (1.0, [1], [-np.inf], True, ok)):
        assert oracle.distill_row(z, None, T, ids, values, rest)["status"] == want
    assert oracle.distill_row(z, np.zeros(5, bool), 1.0, [0], [0.0], False)["status"] \
        == oracle.ROW_EMPTY
    assert oracle.distill_row(np.array([0, np.nan]), None, 1.0, [0], [0.0], False)["status"] \
        == oracle.ROW_NONFINITE
    assert oracle.distill_row(np.full(3, -np.inf), None, 1.0, [0], [0.0], False)["status"] \
        == oracle.ROW_ALL_NEG_INF
    # the student cannot give what the teacher asks for
    assert oracle.distill_row(np.array([0, -np.inf]), None, 1.0, [1], [0.0], False)["loss"] \
        == np.inf


@pytest.mark.parametrize("rest", [False, True])
def test_gradient_formula_against_differences(rest):
    rng = np.random.default_rng(2)
    for _ in range(20):
        V, K, T = 12, int(rng.integers(1, 12)), float(rng.uniform(0.4, 2))
        z = rng.normal(0, 2, V)
        legal = rng.random(V) < 0.8
        legal[0] = True
        ids = rng.permutation(V)[:K]
        values = np.log(rng.dirichlet(np.ones(K + 1))[:K])
        row = oracle.distill_row(z, legal, T, ids, values, rest)
        grad = oracle.distill_grad_row(z, legal, T, ids, values, rest, 1.0, row["state"])
        assert abs(grad.sum()) < 1e-12
        for i in range(V):
            up, down = z.copy(), z.copy()
            up[i] += 1e-6
            down[i] -= 1e-6
            d = (oracle.distill_row(up, legal, T, ids, values, rest)["loss"]
                 - oracle.distill_row(down, legal, T, ids, values, rest)["loss"]) / 2e-6
            assert abs(grad[i] - d) < 1e-7, (i, grad[i], d)


def test_adapted_row_is_the_row_of_the_changed_projection():
    rng = np.random.default_rng(3)
    W, down, up, x = (rng.normal(size=s) for s in ((30, 8), (4, 8), (30, 4), (8,)))
    got = oracle.adapted_row(W @ x, x, down, up, 0.5)
    assert np.allclose(got, (W + 0.5 * up @ down) @ x, rtol=0, atol=1e-12)
    assert np.array_equal(oracle.adapted_row(x, x, None, None, 1.0), x)
