"""The fp64 oracle of the sampler rules, the top log-probs and the distillation loss: closed
forms, invariants, and gradients against central differences."""
import numpy as np
import pytest

from oracle import logits_ops_oracle as lo


def test_rules_on_a_row_done_by_hand():
    x = np.array([[1.0, -2.0, 3.0, 0.5, -1.0, 4.0, 0.0]])
    tokens = np.array([[2, 1, 2, 5, -1, 9, 2]])
    allowed = np.array([[0b1011111]], dtype=np.int32)
    y, _ = lo.process_logits(x, 1, tokens=tokens, hist_len=[7], prompt_len=[2], repetition=[2.0], frequency=[0.5],
                             presence=[0.25], bias_ids=np.array([[3, 3, -1, 99]]),
                             bias=np.array([[7.0, 1.0, 5.0, 5.0]]), allowed=allowed)
    # column 1: prompt only; 2: prompt once, generated twice; 5: generated once, then forbidden
    want = [1.0, -4.0, 1.5 - 1.0 - 0.25, 1.5, -1.0, -np.inf, 0.0]
    assert np.array_equal(y[0], want)
    d = lo.process_logits_bwd(x, np.full((1, 7), 6.0), 1, tokens=tokens, prompt_len=[2], repetition=[2.0],
                              allowed=allowed)
    assert np.array_equal(d[0], [6.0, 12.0, 3.0, 6.0, 6.0, 0.0, 6.0])


def test_rules_gradient_against_differences():
    g = np.random.default_rng(0)
    x = g.normal(size=(3, 40))
    kw = dict(tokens=g.integers(0, 40, (1, 12)), hist_len=[4, 8, 12], prompt_len=[3], repetition=[1.3],
              frequency=[0.4], presence=[0.1], bias_ids=np.array([[1, 7]]), bias=np.array([[2.0, -1.0]]))
    w = g.normal(size=x.shape)
    d = lo.process_logits_bwd(x, w, 3, **kw)
    h = 1e-6
    for r, j in [(0, 0), (1, 7), (2, 1)] + [(2, int(t)) for t in kw["tokens"][0][:4]]:
        e = np.zeros_like(x)
        e[r, j] = h
        num = ((lo.process_logits(x + e, 3, **kw)[0] - lo.process_logits(x - e, 3, **kw)[0]) * w).sum() / (2 * h)
        assert abs(num - d[r, j]) < 1e-7


def test_topk_order_ties_and_rows_without_log_probs():
    x = np.array([[1.0, 3.0, 3.0, -np.inf, -0.0, 0.0], [-np.inf] * 6, [0.0, np.nan, 1, 2, 3, 4]])
    ids, logp, lse = lo.topk_log_softmax(x, 5, 0.5)
    assert ids[0].tolist() == [1, 2, 0, 4, 5]
    assert abs(np.exp(logp[0]).sum() - 1) < 1e-12
    assert ids[1].tolist() == ids[2].tolist() == list(range(5))
    assert np.isnan(logp[1:]).all() and lse[1] == -np.inf and np.isnan(lse[2])


@pytest.mark.parametrize("beta,tail", [(0.0, False), (0.0, True), (0.4, False), (0.4, True), (1.0, True)])
def test_distill_gradient_against_differences_and_invariants(beta, tail):
    g = np.random.default_rng(1)
    R, V, K, T = 3, 50, 6, 0.8
    x = g.normal(size=(R, V)) * 2
    ids = np.stack([g.permutation(V)[:K] for _ in range(R)])
    ids[1, 2] = -1
    t = g.normal(size=(R, V)) * 2
    tl = np.take_along_axis(t - np.log(np.exp(t).sum(1, keepdims=True)), np.maximum(ids, 0), 1)
    w = np.array([1.0, -0.5, 2.0])
    o = lo.distill_topk(x, ids, tl, T, beta, tail, dloss=w)
    assert np.allclose(o["dlogits"].sum(1), 0, atol=1e-12)       # softmax shifts change nothing
    assert np.all(o["loss"] > -1e-12)
    h = 1e-6
    for r, j in [(0, int(ids[0, 0])), (0, 3), (1, int(ids[1, 5])), (2, 11), (2, int(ids[2, 3]))]:
        e = np.zeros_like(x)
        e[r, j] = h
        up, dn = (lo.distill_topk(x + s * e, ids, tl, T, beta, tail)["loss"] for s in (1, -1))
        assert abs(((up - dn) * w).sum() / (2 * h) - o["dlogits"][r, j]) < 1e-7


def test_distill_closed_forms():
    # the student equal to the teacher: no divergence and no gradient, with the rest as a bucket
    g = np.random.default_rng(2)
    x = g.normal(size=(2, 30))
    lp = x - np.log(np.exp(x).sum(1, keepdims=True))
    ids = np.argsort(-x, 1)[:, :5]
    for beta in (0.0, 0.3, 1.0):
        o = lo.distill_topk(x, ids, np.take_along_axis(lp, ids, 1), 1.0, beta, True, dloss=np.ones(2))
        assert np.allclose(o["loss"], 0, atol=1e-12) and np.allclose(o["dlogits"], 0, atol=1e-12)
    # one listed column, renormalised: the cross entropy of that column
    o = lo.distill_topk(x, ids[:, :1], np.full((2, 1), -3.0), 1.0, 0.0, False)
    assert np.allclose(o["loss"], -np.take_along_axis(lp, ids[:, :1], 1)[:, 0])
    # an empty list says nothing
    o = lo.distill_topk(x, np.full((2, 3), -1), np.zeros((2, 3)), 1.0, 0.0, True, dloss=np.ones(2))
    assert np.allclose(o["loss"], 0) and np.allclose(o["dlogits"], 0, atol=1e-15)
    # a column listed twice, a column past the vocabulary
    o = lo.distill_topk(x, np.array([[3, 3], [1, 30]]), np.full((2, 2), -1.0), 1.0, 0.0, True, dloss=np.ones(2))
    assert np.isnan(o["loss"]).all() and np.isnan(o["dlogits"]).all()
