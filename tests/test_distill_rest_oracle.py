"""The fp64 oracle of the distillation where nothing is left outside the teacher's list."""
import numpy as np
import pytest

from oracle import logits_ops_oracle as lo


@pytest.mark.parametrize("beta", [0.0, 0.3, 1.0])
def test_a_student_equal_to_its_teacher_has_no_loss_when_everything_is_listed(beta):
    x = np.random.default_rng(0).normal(size=(3, 7)) * 2
    lp = x - np.log(np.exp(x).sum(1, keepdims=True))
    ids = np.tile(np.arange(7), (3, 1))
    o = lo.distill_topk(x, ids, lp, 1.0, beta, True, dloss=np.ones(3))
    assert np.allclose(o["loss"], 0, atol=1e-12) and np.allclose(o["dlogits"], 0, atol=1e-12)
    assert np.all(o["p_rest"] == 0)


@pytest.mark.parametrize("beta", [0.0, 0.3, 1.0])
def test_without_a_rest_the_tail_changes_nothing(beta):
    """Columns outside the list at -inf: any shift of the teacher's log-probs gives the same, and for
    beta < 1 so does the form without a tail; the gradient agrees with differences."""
    g = np.random.default_rng(1)
    x = np.full((2, 40), -np.inf)
    ids = np.stack([g.permutation(40)[:5] for _ in range(2)])
    np.put_along_axis(x, ids, g.normal(size=(2, 5)), 1)
    lp = g.normal(size=(2, 5))
    w = np.array([1.0, -0.5])
    o = lo.distill_topk(x, ids, lp, 0.8, beta, True, dloss=w)
    assert np.all(np.isfinite(o["loss"])) and np.all(o["loss"] > 0) and np.allclose(o["dlogits"].sum(1), 0, atol=1e-12)
    shifted = lo.distill_topk(x, ids, lp - 0.7, 0.8, beta, True, dloss=w)
    assert np.allclose(shifted["loss"], o["loss"]) and np.allclose(shifted["dlogits"], o["dlogits"])
    if beta < 1.0:
        assert np.allclose(lo.distill_topk(x, ids, lp, 0.8, beta, False)["loss"], o["loss"])
    for r, k in ((0, 0), (1, 3)):
        e = np.zeros_like(x)
        e[r, ids[r, k]] = 1e-6
        up, dn = (lo.distill_topk(x + s * e, ids, lp, 0.8, beta, True)["loss"] for s in (1, -1))
        assert abs(((up - dn) * w).sum() / 2e-6 - o["dlogits"][r, ids[r, k]]) < 1e-7


def test_one_unlisted_column_is_a_rest():
    x = np.full((1, 9), -np.inf)
    x[0, :4] = [1.0, 0.5, 0.0, -40.0]
    ids, lp = np.array([[0, 1, 2]]), np.log(np.array([[0.5, 0.3, 0.2]]))
    o = lo.distill_topk(x, ids, lp, 1.0, 0.0, True)
    assert np.isfinite(o["loss"][0]) and 0 < o["p_rest"][0] < 1e-16
    q = np.array([0.5, 0.3, 0.2, lo.REST_MIN])
    p = np.exp(x[0, :4]) / np.exp(x[0, :4]).sum()
    assert abs(o["loss"][0] - (q * np.log(q / p)).sum()) < 1e-12
