"""Accuracy of the distillation where a small quantity is a difference of larger ones."""
import numpy as np
import pytest
import torch

from logits_ops_util import DEV, f64, randn
from oracle import logits_ops_oracle as lo
from rl_fine_tuning_pass_gb300 import binding as rp
from test_distill_topk_gpu import EPS, check

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


@pytest.mark.parametrize("beta", [0.1, 1e-3, 1e-5, 1e-8, 0.9, 0.999, 1 - 2.0 ** -16])
@pytest.mark.parametrize("tail", [False, True])
def test_gradients_of_mixtures_relative_to_the_smaller_weight(beta, tail):
    """With w the smaller of the weights, each bucket's G is w times something of the order of
    (p + q)(1 + |log q/p|).  p is within EPS of itself and log q/p within 2 EPS (test_distill_topk_gpu.py),
    so G is within w 4 EPS (p + q)(1 + |log q/p|) =: E; the gradient of a listed column is
    g (G - p S), of another g p (G_rest / p_rest - S), S the sum of all G."""
    R, V, K, T = 8, 700, 9, 1.0
    x = randn(1, R, V, seed=1)
    ids = torch.stack([torch.randperm(V, generator=torch.Generator().manual_seed(r))[:K] for r in range(R)])
    for r in range(R):      # gaps of both signs between student and teacher
        x[0, r, ids[r]] += torch.linspace(-2.5 * r, 2.5 * r, K)
    lp = torch.log_softmax(randn(R, K + 1, seed=2), 1)[:, :K].contiguous()
    w, b = torch.ones(R), float(np.float32(beta))
    xs = f64(x)
    o = lo.distill_topk(xs, ids.numpy(), lp.numpy(), T, b, tail, None, np.ones(R))
    p = np.exp(xs - o["lse"][:, None])
    at = ids.numpy()
    P = np.concatenate([np.take_along_axis(p, at, 1), o["p_rest"][:, None]], 1)
    q = np.exp(lp.double().numpy())
    Q = np.concatenate([q, 1 - q.sum(1, keepdims=True)], 1) if tail else \
        np.concatenate([q / q.sum(1, keepdims=True), np.zeros((R, 1))], 1)
    with np.errstate(divide="ignore"):
        ratio = np.where(Q > 0, np.abs(np.log(Q / P)), 0.0)
    E = min(b, 1 - b) * 4 * EPS * (P + Q) * (1 + ratio)
    ES = E.sum(1, keepdims=True)
    tol = p * (E[:, -1:] / P[:, -1:] + 2 * ES)
    np.put_along_axis(tol, at, E[:, :-1] + 2 * np.take_along_axis(p, at, 1) * ES, 1)
    # (p S besides: p is within EPS, and |S| within the sum of |G| <= ES / (4 EPS))
    tol = tol + EPS * p * ES / (4 * EPS) + 2.0 ** -23 * np.abs(o["dlogits"]) + 2.0 ** -126
    d = lambda t: t.to(DEV)  # noqa: E731
    how = dict(T=T, beta=b, tail=tail)
    f = rp.distill_topk_fwd(d(x), d(ids), d(lp), **how)
    dl = rp.distill_topk_bwd(d(x), d(ids), d(lp), d(w), f["lse"], f["p_rest"], **how)
    u = rp.distill_topk_fused(d(x), d(ids), d(lp), d(w), **how)
    for name, got in (("backward", dl), ("fused", u["dlogits"])):
        off = np.abs(f64(got) - o["dlogits"]) - tol
        assert off.max() <= 0, f"{name}: {int((off > 0).sum())} outside, worst {off.max() / min(b, 1 - b):.3g} of the weight"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("beta", [0.0, 0.5])
@pytest.mark.parametrize("shift", [-300.0, -20.0, 60.0])
def test_a_shifted_teacher_is_the_same(dtype, beta, shift):
    """Without the tail the teacher is renormalised: a shift of its log-probs, as fp32 holds them,
    changes nothing; also where a student's rest has no mass and the tail is asked for."""
    V, K = 203, 30
    x = (randn(1, 6, V, seed=4) * 12).to(dtype)
    x[0, 4:] = float("-inf")
    x[0, 4:, 50:50 + K] = (randn(2, K, seed=6) * 12).to(dtype)
    ids = torch.arange(50, 50 + K).repeat(6, 1)
    lp = torch.log_softmax(randn(6, K, seed=5), 1) + shift
    check(x.to(DEV), ids, lp, 1.0, beta, False, what=f"shift {shift}")
    if shift < 0:
        check(x[:, 4:].to(DEV), ids[4:], lp[4:], 1.0, beta, True, what=f"no rest, shift {shift}")
