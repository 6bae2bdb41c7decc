"""The oracle of the distillation loss against its closed forms, its gradient against
differences."""
import math

import numpy as np
import pytest

import oracle as O


def kl(q, p):
    return float(np.sum(q[q > 0] * np.log(q[q > 0] / p[q > 0])))


def softmax(z):
    e = np.exp(z - np.max(z))
    return e / e.sum()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T", [1.0, 2.5, 0.3])
def test_against_the_definition(T, tail):
    r = np.random.default_rng(3)
    z, t = r.standard_normal(30) * 2, softmax(r.standard_normal(30) * 2)
    ids = np.argsort(-t)[:6]
    lp = np.log(t[ids])
    loss, grad, _ = O.distill.row(z, ids, lp, T, tail)
    p = softmax(z / T)
    if tail:
        q = np.append(t[ids], 1 - t[ids].sum())
        ref = kl(q, np.append(p[ids], 1 - p[ids].sum()))
        assert 0 < ref <= kl(t, p) + 1e-15
    else:
        q = softmax(lp / T)
        ref = kl(q, p[ids])
    assert math.isclose(loss, ref, rel_tol=1e-12)
    for i in range(30):
        h = np.zeros(30)
        h[i] = 1e-5
        d = (O.distill.row(z + h, ids, lp, T, tail)[0] - O.distill.row(z - h, ids, lp, T, tail)[0]) / 2e-5
        assert abs(d - grad[i]) <= 1e-8
    assert abs(grad.sum()) < 1e-12


def test_the_teacher_itself_has_loss_and_gradient_zero():
    z = np.random.default_rng(4).standard_normal(50)
    lp = np.log(softmax(z))
    ids = np.argsort(-z)[:5]
    loss, grad, _ = O.distill.row(z, ids, lp[ids], 1.0, True)
    assert abs(loss) < 1e-14 and np.max(np.abs(grad)) < 1e-15
    assert math.isclose(O.distill.row(z, ids, lp[ids])[0], -math.log(np.exp(lp[ids]).sum()), rel_tol=1e-12)


def test_rows_and_entries_that_are_not_there():
    z = np.array([0.0, 1.0, 2.0, np.nan])
    assert O.distill.row(z, [-1, -1], [0, 0])[0] == 0.0
    assert math.isnan(O.distill.row(z, [0, -1], [0, 0])[0])
    assert math.isnan(O.distill.row(z[:3], [0, 3], [0, 0])[0])
    a, b = O.distill.row(z[:3], [2, -1], [-1.0, 5.0]), O.distill.row(z[:3], [2], [-1.0])
    assert a[0] == b[0] and (a[1] == b[1]).all()
    assert (O.distill.row(z, [0, 1], [0, 0], weight=0.0)[1] == 0).all()
    # a token listed twice with halves of a probability: the terms differ by its log 2
    one = O.distill.row(z[:3], [2, 0], [math.log(0.5), math.log(0.25)], 1.0, True)
    two = O.distill.row(z[:3], [2, 0, 2], [math.log(0.25), math.log(0.25), math.log(0.25)], 1.0, True)
    assert math.isclose(one[0] - two[0], 0.5 * math.log(2), rel_tol=1e-12) and np.allclose(one[1], two[1], atol=1e-16)


def test_probabilities_of_zero():
    z = np.array([0.0, -np.inf, 1.0, -np.inf])
    assert O.distill.row(z, [1, 2], [math.log(0.5), math.log(0.5)])[0] == math.inf
    assert math.isfinite(O.distill.row(z, [1, 2], [-math.inf, 0.0])[0])
    assert O.distill.row(z, [0, 2], [math.log(0.5), math.log(0.25)], 1.0, True)[0] == math.inf
    assert math.isnan(O.distill.row(np.full(3, -np.inf), [1], [0.0])[0])
    assert math.isnan(O.distill.row(z, [0, 2], [-math.inf, -math.inf])[0])
